"""Sizes of the 8-bit operands and workspaces up to the largest accepted shapes: each is at least the sum of its parts, or the shape is
refused.  Nothing is launched, so the sizes need no memory behind them."""
import pytest

from bit_expert_ffn_moe_gb300 import binding as B

MOST = 2 ** 28  # rows at most
CONTROL = 8192


def rows_bytes(room, K):
    """What the rows' layout takes: fp16 numbers [ceil(K / 64)][room][64] and fp32 scales [room]."""
    return -(-K // 64) * room * 128 + 4 * room


def room_of(M, E):
    return -(-M // 8) * 8 + 8 * E + 16


@pytest.mark.parametrize("M,K", [(MOST, 1), (MOST, 16), (MOST, 64), (MOST, 4096), (MOST - 1, 4096), (MOST - 15, 16), (MOST - 16, 16), (MOST - 17, 16),
                                 (MOST - 24, 64), (2 ** 23, 131072), (2 ** 23 - 1, 131072), (2 ** 23 - 16, 131072), (2 ** 23 - 17, 131072),
                                 (2 ** 26, 2 ** 14), (2 ** 26 - 9, 2 ** 14)])
def test_a_workspace_has_room_for_the_rows(M, K):
    for N in (1, 2 ** 12 if M == MOST else 2):
        size = B.moe_int8_workspace_size(M, N, K)
        assert size >= CONTROL + rows_bytes(room_of(M, 0), K), (M, N, K, size)


def test_shapes_beyond_are_refused():
    for M, N, K in ((MOST + 1, 1, 16), (MOST, 1, 4097), (2 ** 23 + 1, 1, 131072), (2 ** 26 + 1, 1, 2 ** 14), (MOST, 4097, 16)):
        assert B.moe_int8_workspace_size(M, N, K) == 0, (M, N, K)


@pytest.mark.parametrize("T,k,E", [(2 ** 23, 32, 1024), (2 ** 23 - 1, 32, 1024), (2 ** 28 - 8200, 1, 1024), (2 ** 28 - 8208, 1, 1024), (2 ** 28 - 8209, 1, 1024),
                                   (2 ** 28, 1, 1), (2 ** 28 - 23, 1, 1), (2 ** 28 - 24, 1, 1)])
@pytest.mark.parametrize("d,I", [(16, 8), (64, 70), (1024, 512), (1, 1)])
def test_a_sparse_layers_workspace_has_room_for_both_rows(T, k, E, d, I):  # noqa: E741
    P = T * k
    for dtype, width in ((B.MOE_BF16, 2), (B.MOE_F32, 4)):
        size = B.moe_int8_experts_workspace_size(T, d, E, k, I, dtype)
        room = room_of(P, E)
        assert size >= CONTROL + rows_bytes(room, d) + rows_bytes(room, I) + width * P * (d + I) + 4 * P + 4 * (E + 1), (T, k, E, d, I, size)


@pytest.mark.parametrize("M,E,K", [(0, 0, 1), (0, 1024, 1), (1, 0, 64), (1000, 7, 65), (MOST, 0, 16), (MOST, 1024, 16), (MOST - 9, 1024, 4096),
                                   (2 ** 23, 0, 131072), (2 ** 23, 1024, 131072)])
def test_the_bytes_of_the_rows_of_every_room(M, E, K):
    room = B.moe_int8_rows_room(M, E)
    assert room == room_of(M, E) and room % 8 == 0
    assert B.moe_int8_rows_bytes(room, K) == rows_bytes(room, K) - 4 * room


def test_no_bytes_for_rooms_that_no_shape_has():
    for room, K in ((-8, 64), (MOST + 8 * 1024 + 24, 64), (2 ** 40, 64), (2 ** 62, 131072), (2 ** 24, 131072), (32, 0), (32, -1), (32, 131073)):
        assert B.moe_int8_rows_bytes(room, K) == 0, (room, K)

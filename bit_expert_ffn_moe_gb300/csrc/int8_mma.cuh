// int8_mma.cuh -- what the 8-bit products on the tensor cores are made of: fp16 products with the weights in tensor memory, the
// conversion of the weights, copies and barriers.
#pragma once

#include "int8_common.cuh"
#include "tcgen05.cuh"

namespace moe {

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Arrive on the barrier at this place in CTA 0 of the cluster.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\t"
        "mapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void arrive(uint64_t* bar) {
    if constexpr (PAIR) arrive_leader(bar);
    else mbar_arrive(bar);
}
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .b16 both;\n\t"
            "mov.b16 both, 3;\n\t"
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], both;\n\t}" ::"r"(smem_u32(bar))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A step's four products of 16 values: A from tensor memory (8 columns each), B 32 bytes further along its rows each.
template <bool PAIR>
__device__ __forceinline__ void step_products(uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
    constexpr uint32_t kHigh = (1024 >> 4) | (1u << 14) | (2u << 29);  // of desc_sw128
#define MOE_PRODUCT(group, i, pred)                                                     \
    "add.u32 c, %1, 8*" #i ";\n\tadd.u32 l, %2, 2*" #i ";\n\tmov.b64 t, {l, %5};\n\t" \
    "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [c], t, %3, " pred ";\n\t"
#define MOE_STEP(group)                                                                                                       \
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 c, l;\n\t.reg .b64 t;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t" \
                 MOE_PRODUCT(group, 0, "p") MOE_PRODUCT(group, 1, "q") MOE_PRODUCT(group, 2, "q") MOE_PRODUCT(group, 3, "q") "}" ::"r"(d), \
                 "r"(a), "r"(b_low), "r"(idesc), "r"(accumulate), "n"(kHigh)                                                  \
                 : "memory")
    if constexpr (PAIR) MOE_STEP("2");
    else MOE_STEP("1");
#undef MOE_STEP
#undef MOE_PRODUCT
}

// Four whole numbers of eight bits as fp16: with 128 added they are the last eight bits of numbers from 1024 on.
__device__ __forceinline__ void to_fp16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u, bias = 0x64806480u;  // 1024 + 128, twice
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
        "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// This thread's row of a tile of weights (w: its first 16 bytes) as fp16.
__device__ __forceinline__ void convert_row(const unsigned char* w, uint32_t (&h)[32]) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(w + j * 2048);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        to_fp16(v[j].x, h[8 * j], h[8 * j + 1]);
        to_fp16(v[j].y, h[8 * j + 2], h[8 * j + 3]);
        to_fp16(v[j].z, h[8 * j + 4], h[8 * j + 5]);
        to_fp16(v[j].w, h[8 * j + 6], h[8 * j + 7]);
    }
}
// Instruction descriptor of kind::f16: A and B fp16, K-major, D fp32, shape M x N.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
// A place in a ring of `size`, and how often it has gone round, modulo 2.
struct Turn {
    const int size;
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ explicit Turn(int n) : size(n) {}
    __device__ __forceinline__ void next() {
        if (++at == size) at = 0, parity ^= 1;
    }
};
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}


}  // namespace moe

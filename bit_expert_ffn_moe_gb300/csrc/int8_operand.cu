// int8_operand.cu -- operands of the 8-bit products.  A row v of K numbers is held as whole numbers q and one fp32 scale s:
//   s = max |v| / 127 (1 for a row of zeros),  q = v / s rounded to the nearest whole number, ties to even, within -127 .. 127
// (each step rounded to fp32).  A row with a NaN or an infinity gets s = NaN and q = 0, which makes its results NaN.
// Layouts: ops.cuh.  Weights are kept in one byte each; activations as fp16 numbers, which is what the tensor cores take
// (sm_103a's have no 8-bit whole numbers), in the layout that they read, so that a product's copies are contiguous.
#include "int8_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kKept = 4;  // pieces of 8 values that a thread keeps between the two passes over its row (256 threads: 8192 values)

// The largest of a row's magnitudes over the `warps` warps that share it (all of them call this).
__device__ __forceinline__ uint32_t most_of(uint32_t m, int warps, uint32_t* part) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (warps == 1) {
        __syncwarp();
        return m;
    }
    const int warp = threadIdx.x >> 5, first = warp / warps * warps;
    if ((threadIdx.x & 31) == 0) part[warp] = m;
    __syncthreads();
    for (int i = 0; i < warps; ++i) m = max(m, part[first + i]);
    return m;
}

// The expert whose rows hold row r < offsets[E]: the last e with offsets[e] <= r.
__device__ __forceinline__ int expert_of(const int32_t* offsets, int E, int r) {
    int lo = 0, hi = E;  // offsets[lo] <= r < offsets[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (offsets[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// `warps` warps of a CTA share a row; it is read once into registers (its first kKept pieces per thread; what is longer is read
// again), quantised, and written to the rows that it goes to.  Bound by the writing of k rows in 16 bits; for few rows by its chain of
// loads, so the row's, the offsets' and its places' are all in flight together.  4096 x 8192 in bf16: 29.3 us (4.6 TB/s), in fp32 34.4 us
// (5.9 TB/s), to 8 rows each 98 us (6.2 TB/s); 16 x 4096: 2.2 us.  Wide loads of 16-bit numbers run with 5 CTAs on an SM (48 registers; with
// 4, 31.2 us); fp32 with 4, since 48 registers do not hold its pieces (with 5, 45.0 us), and so do loads of single numbers (2000 x 1543 in
// bf16: 6.8 us with 4, 7.6 with 5).
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, WIDE && sizeof(T) == 2 ? 5 : 4) int8_rows_kernel(const Int8RowsArgs a, const int warps) {
    __shared__ uint32_t part[kThreads / 32];
    __shared__ int64_t to_smem[kThreads / 32][kMaxK];
    extern __shared__ int32_t offsets[];  // [E + 1]
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = kThreads / 32 / warps, mine = warp / warps;
    const int64_t t = (int64_t)blockIdx.x * rows + mine;
    const int first = threadIdx.x - mine * warps * 32, step = warps * 32;
    const int k = a.inv ? a.k : 1;
    const bool live = t < a.T, places = warp % warps == 0 && lane < k && live;
    const T* x = static_cast<const T*>(a.x) + t * a.ld;
    const int pieces = (int)((a.K + 63) / 64 * 8);
    int64_t r = t;
    if (places && a.inv) r = __ldg(a.inv + t * k + lane);
    Eight<T> kept[kKept];
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
        if (live && first + i * step < pieces) kept[i].template load<WIDE>(x, 8 * (int64_t)(first + i * step), a.K);
        else kept[i].clear();
    }
    if (a.offsets) {
        for (int e = threadIdx.x; e <= a.E; e += kThreads) offsets[e] = __ldg(a.offsets + e);
        __syncthreads();
    }
    if (places) {  // where the row goes
        int64_t to = r;
        if (a.offsets) {
            to = -1;
            if (r >= 0 && r < offsets[a.E]) {
                const int e = expert_of(offsets, a.E, (int)r);
                to = int8_first_row(offsets[e], e) + r - offsets[e];
            }
        }
        to_smem[mine][lane] = to < a.room ? to : -1;
    }
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < kKept; ++i) most = kept[i].most(most);
    if (live)
        for (int c = first + kKept * step; c < pieces; c += step) {
            Eight<T> v;
            v.template load<WIDE>(x, 8 * (int64_t)c, a.K);
            most = v.most(most);
        }
    const Scale s = scale_of(most_of(Eight<T>::as_fp32(most), warps, part));  // (and the places are there)
    if (!live) return;
    if (first < k && to_smem[mine][first] >= 0) a.s[to_smem[mine][first]] = s.s;
    auto put = [&](int c, const Eight<T>& x8) {
        float v[8], q[8];
        x8.get(v);
        whole8(v, s, q);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(q[2 * i], q[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        for (int j = 0; j < k; ++j) {
            const int64_t to = to_smem[mine][j];
            if (to >= 0)
                *reinterpret_cast<uint4*>(a.q + ((int64_t)(c / 8) * a.room + to) * 64 + ((c % 8) ^ (int)(to % 8)) * 8) =
                    make_uint4(o[0], o[1], o[2], o[3]);
        }
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i)
        if (first + i * step < pieces) put(first + i * step, kept[i]);
    for (int c = first + kKept * step; c < pieces; c += step) {
        Eight<T> v;
        v.template load<WIDE>(x, 8 * (int64_t)c, a.K);
        put(c, v);
    }
}

// One CTA per row of weights; a thread puts 16 neighbouring values together by single loads.  Done once for a weight, so it was left at that:
// 128 x 4096 x 8192 (4.3 G values) laid out from int8 in 3.4 ms (2.5 TB/s), quantised from bf16 in 6.2 ms (2.1 TB/s); one matrix of
// these 32 and 56 us.  INT8: the numbers as they are given.
template <typename T>
__global__ void __launch_bounds__(kThreads) int8_pack_kernel(const Int8PackArgs a) {
    constexpr bool kWhole = sizeof(T) == 1;
    __shared__ uint32_t part[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;  // of E * rows
    const int64_t e = row / a.rows, n = a.first + a.step * (row - e * a.rows);
    const T* w = static_cast<const T*>(a.w) + row * a.ld;
    const int64_t KT = (a.K + 63) / 64;
    Scale s = {};
    if constexpr (!kWhole) {
        uint32_t most = 0;
        for (int64_t c = threadIdx.x; c < a.K; c += kThreads) most = max(most, magnitude(value<T>(w[c])));
        s = scale_of(most_of(most, kThreads / 32, part));
    }
    if (threadIdx.x == 0) a.s[e * a.N + n] = kWhole ? a.s_in[row] : s.s;
    uint8_t* q = a.q + e * int8_tiles(a.N, a.K) * kInt8Tile + (n / 128) * KT * kInt8Tile + (n % 128) * 16;
    for (int64_t c = threadIdx.x; c < 4 * KT; c += kThreads) {
        uint32_t o[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int64_t at = 16 * c + i;
            int b = 0;
            if (at < a.K) {
                if constexpr (kWhole) b = w[at];
                else b = (int)whole(value<T>(w[at]), s.s, s.bad);
            }
            o[i / 4] |= (uint32_t)(b & 255) << (8 * (i % 4));
        }
        *reinterpret_cast<uint4*>(q + (c / 4) * kInt8Tile + (c % 4) * 2048) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <typename T>
cudaError_t launch_rows(Int8RowsArgs a, cudaStream_t st) {
    const int pieces = (int)((a.K + 63) / 64 * 8);
    // warps for a row: so many that they keep it; of few rows more, down to a piece a thread
    int warps = 1;
    while (warps < kThreads / 32 && (warps * 32 * kKept < pieces || (warps * 32 < pieces && a.T * warps < (int64_t)sm_count() * 8))) warps *= 2;
    const int64_t rows = kThreads / 32 / warps;
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ld * (int64_t)sizeof(T)) % 16 == 0;
    const void* f = wide ? (const void*)int8_rows_kernel<T, true> : (const void*)int8_rows_kernel<T, false>;
    void* args[] = {&a, &warps};
    const size_t smem = a.offsets ? sizeof(int32_t) * (size_t)(a.E + 1) : 0;
    return launch_kernel(f, dim3((unsigned)((a.T + rows - 1) / rows)), dim3(kThreads), smem, st, true, args);
}

}  // namespace

cudaError_t launch_int8_rows(const Int8RowsArgs& a, moe_dtype dtype, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    switch (dtype) {
        case MOE_F32: return launch_rows<float>(a, st);
        case MOE_BF16: return launch_rows<__nv_bfloat16>(a, st);
        default: return launch_rows<__half>(a, st);
    }
}

cudaError_t launch_int8_pack(const Int8PackArgs& a, int dtype, cudaStream_t st) {
    if (a.E == 0 || a.rows == 0) return cudaSuccess;
    const void* f = dtype < 0             ? (const void*)int8_pack_kernel<int8_t>
                    : dtype == MOE_F32    ? (const void*)int8_pack_kernel<float>
                    : dtype == MOE_BF16   ? (const void*)int8_pack_kernel<__nv_bfloat16>
                                          : (const void*)int8_pack_kernel<__half>;
    void* args[] = {const_cast<Int8PackArgs*>(&a)};
    return launch_kernel(f, dim3((unsigned)(a.E * a.rows)), dim3(kThreads), 0, st, true, args);
}

}  // namespace moe

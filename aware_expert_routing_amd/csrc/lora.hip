// Projections shared by a batch with low-rank adapters of its requests, and
// the shared expert built from three of them.
//
//   y_i = W x_i + s_a B_a (A_a x_i),   a = the adapter of token i (or none)
//
// W and A_a are packed bf16 tiles of 16 rows x 32 columns (pack.hip), so one
// wave load of 1 KB is the A operand of v_mfma_f32_16x16x32_bf16; B_a is
// packed in half tiles of 16 rows x 16 ranks, the A operand of
// v_mfma_f32_16x16x16_bf16.  The two meet without a shuffle: the first
// product's C layout (lane = 16 q + n holds ranks 4 q .. 4 q + 3 of token n)
// is the second's B operand layout.
//
// Two launches: `shrink` forms v_i = s_a A_a x_i in fp32, and the projection
// adds B_a v_i to its accumulators before it stores.
//
// Precision: products are bf16 x bf16 with fp32 sums.  An fp32 value enters as
// three bf16 terms cut from its 24 significant bits (exact); v enters an fp32
// output the same way and a bf16 output as two terms (16 bits, against the
// output's 8).
#include "internal.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int kWave = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma32(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}
__device__ __forceinline__ f32x4 mma16(u32x2 a, u32x2 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0,
                                                     0, 0);
}

// The leading 8 significant bits of f as a float, and what is left (0 for an
// infinity, whose difference to itself is NaN).
__device__ __forceinline__ float cut8(float f, float& rest) {
    const float t = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
    const float r = f - t;
    rest = r == r ? r : 0.0f;
    return t;
}
__device__ __forceinline__ uint32_t pair_hi(float a, float b) {   // bf16 bits of a (low half) and b
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// f (P pairs) as T bf16 terms, largest first.
template <int T, int P>
__device__ __forceinline__ void split(const float (&f)[2 * P], uint32_t (&t)[T][P]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float a = f[2 * p], b = f[2 * p + 1];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            float ra, rb;
            const float ta = cut8(a, ra), tb = cut8(b, rb);
            t[i][p] = pair_hi(ta, tb);
            a = ra;
            b = rb;
        }
    }
}

// One activation fragment: lane (n = l % 16, q = l / 16) holds columns
// c .. c + 7 of its token, as the bf16 terms that enter the product.
template <typename XT>
struct Frag;
template <>
struct Frag<uint16_t> {
    static constexpr int kTerms = 1;
    u32x4 raw;
    __device__ void load(const uint16_t* p) { raw = *reinterpret_cast<const u32x4*>(p); }
    __device__ void terms(u32x4 (&t)[1]) const { t[0] = raw; }
};
template <>
struct Frag<float> {
    static constexpr int kTerms = 3;
    f32x4 lo, hi;
    __device__ void load(const float* p) {
        lo = *reinterpret_cast<const f32x4*>(p);
        hi = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ void terms(u32x4 (&t)[3]) const {
        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t s[3][4];
        split<3, 4>(f, s);
#pragma unroll
        for (int i = 0; i < 3; ++i) t[i] = u32x4{s[i][0], s[i][1], s[i][2], s[i][3]};
    }
};

__device__ __forceinline__ int real_tokens(const ProjArgs& a) {
    return a.n_valid != nullptr ? min(max(*a.n_valid, 0), a.B) : a.B;
}
// The adapter of token i (lane-wise), -1 where there is none.
__device__ __forceinline__ int adapter_of(const ProjArgs& a, int i, int B_real) {
    if (a.adapter == nullptr || i >= B_real) return -1;
    const int id = a.adapter[i];
    return (id >= 0 && id < a.n_adapters) ? id : -1;
}
// Rank blocks of 16 that adapter `h` contributes (an adapter wider than the
// call's max_rank contributes nothing: its v has no room).
__device__ __forceinline__ int rank_blocks(const moe_lora_handle& h, int max_rank) {
    return (h.rank > 0 && h.rank <= max_rank) ? h.rank / 16 : 0;
}

// ---------------------------------------------------------------------------
// shrink: v[i, r] = scale * sum_h A[r, h] x[i, h].  One workgroup per (token
// of a tile of 16 that is the first with its adapter, rank block, table); its
// four waves split H and add their sums in LDS in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 4;

template <typename XT>
__global__ __launch_bounds__(kShrinkWaves * kWave) void shrink_kernel(ProjArgs a) {
    __shared__ f32x4 part[kShrinkWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int i0 = (blockIdx.x >> 4) * 16, slot = blockIdx.x & 15;
    const int B_real = real_tokens(a);
    const moe_lora_handle* table = a.table[blockIdx.z];
    if (i0 + slot >= B_real || table == nullptr) return;
    const int id = adapter_of(a, i0 + n, B_real);
    const int ad = __builtin_amdgcn_readlane(id, slot);
    if (ad < 0) return;
    const uint64_t same = __ballot(id == ad) & 0xffffull;
    if (__ffsll(static_cast<unsigned long long>(same)) - 1 != slot) return;
    const moe_lora_handle h = table[ad];
    const int rb = blockIdx.y;
    if (rb >= rank_blocks(h, a.max_rank)) return;

    const int S = a.H / 32;
    const char* A = static_cast<const char*>(h.a) + (static_cast<size_t>(rb) * S) * 1024 + lane * 16;
    const XT* x = static_cast<const XT*>(a.x) + static_cast<size_t>(min(i0 + n, B_real - 1)) * a.H + 8 * q;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = wave; s < S; s += kShrinkWaves) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(A + static_cast<size_t>(s) * 1024);
        Frag<XT> f;
        f.load(x + s * 32);
        u32x4 t[Frag<XT>::kTerms];
        f.terms(t);
#pragma unroll
        for (int k = Frag<XT>::kTerms - 1; k >= 0; --k) acc = mma32(w, t[k], acc);
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0 || id != ad) return;
    f32x4 v = part[0][lane];
#pragma unroll
    for (int w = 1; w < kShrinkWaves; ++w) v += part[w][lane];
    float* out = a.v[blockIdx.z] + static_cast<size_t>(i0 + n) * a.max_rank + 16 * rb + 4 * q;
    *reinterpret_cast<f32x4*>(out) = v * h.scale;
}

// Adds the adapters' part to the accumulator of row block ob and the 16
// tokens whose adapters are `id` (lane 16 q + n: token n); v_row is the lane's
// token's row of v.
template <int VT>
__device__ __forceinline__ f32x4 expand(const ProjArgs& a, int m, int ob, int id, const float* v_row, f32x4 acc) {
    const int lane = threadIdx.x & (kWave - 1), q = lane >> 4;
    const moe_lora_handle* table = a.table[m];
    if (table == nullptr) return acc;
    uint32_t rem = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
    while (rem != 0u) {
        const int ad = __builtin_amdgcn_readlane(id, __ffs(rem) - 1);
        const bool mine = id == ad;
        rem &= ~static_cast<uint32_t>(__ballot(mine));
        const moe_lora_handle h = table[ad];
        const int nb = rank_blocks(h, a.max_rank);
        const char* b = static_cast<const char*>(h.b) + (static_cast<size_t>(ob) * nb) * 512 + lane * 8;
        for (int r = 0; r < nb; ++r) {
            const u32x2 bw = *reinterpret_cast<const u32x2*>(b + r * 512);
            float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (mine) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(v_row + 16 * r + 4 * q);
                f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
            }
            uint32_t t[VT][2];
            split<VT, 2>(f, t);
#pragma unroll
            for (int k = VT - 1; k >= 0; --k) acc = mma16(bw, u32x2{t[k][0], t[k][1]}, acc);
        }
    }
    return acc;
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + __expf(-z)); }

// Four consecutive outputs of one token.
__device__ __forceinline__ void store4(float* p, f32x4 v, int accumulate) {
    if (accumulate) v += *reinterpret_cast<const f32x4*>(p);
    *reinterpret_cast<f32x4*>(p) = v;
}
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v, int) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<u32x2*>(p) = __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
}

// ---------------------------------------------------------------------------
// Streaming projection: a workgroup owns RB row blocks of 16 outputs (of NM
// matrices: 2 = gate and up, whose result is silu(g) u) and NT tiles of 16
// tokens; its W waves take the columns' tiles in turn and add their sums in
// LDS in a fixed order.
// ---------------------------------------------------------------------------
template <typename XT, typename YT, int NM, int NT, int RB, int W>
__global__ __launch_bounds__(W* kWave) void proj_stream_kernel(ProjArgs a) {
    constexpr int VT = sizeof(YT) == 4 ? 3 : 2;
    constexpr int TT = Frag<XT>::kTerms;
    __shared__ f32x4 part[W][NM * RB * NT][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int B_real = real_tokens(a);
    const int i0 = blockIdx.y * 16 * NT;
    if (i0 >= B_real) return;
    const int ob0 = blockIdx.x * RB, blocks = a.O / 16;
    const int S = a.H / 32;

    const char* wp[NM][RB];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
            wp[m][r] = static_cast<const char*>(a.w[m]) + (static_cast<size_t>(min(ob0 + r, blocks - 1)) * S) * 1024 +
                       lane * 16;
    const XT* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        xp[t] = static_cast<const XT*>(a.x) + static_cast<size_t>(min(i0 + 16 * t + n, B_real - 1)) * a.H + 8 * q;

    f32x4 acc[NM][RB][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
    for (int s = wave; s < S; s += W) {
        u32x4 w[NM][RB];
        Frag<XT> f[NT];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int r = 0; r < RB; ++r) w[m][r] = *reinterpret_cast<const u32x4*>(wp[m][r] + static_cast<size_t>(s) * 1024);
#pragma unroll
        for (int t = 0; t < NT; ++t) f[t].load(xp[t] + s * 32);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            u32x4 x[TT];
            f[t].terms(x);
#pragma unroll
            for (int k = TT - 1; k >= 0; --k)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < RB; ++r) acc[m][r][t] = mma32(w[m][r], x[k], acc[m][r][t]);
        }
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) part[wave][(m * RB + r) * NT + t][lane] = acc[m][r][t];
    __syncthreads();
    for (int p = wave; p < RB * NT; p += W) {
        const int r = p / NT, t = p % NT;
        const int ob = ob0 + r, i = i0 + 16 * t + n;
        if (ob >= blocks || i0 + 16 * t >= B_real) continue;
        const int id = adapter_of(a, i, B_real);
        f32x4 sum[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sum[m] = part[0][m * RB * NT + p][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum[m] += part[w][m * RB * NT + p][lane];
            sum[m] = expand<VT>(a, m, ob, id, a.v[m] + static_cast<size_t>(min(i, B_real - 1)) * a.max_rank, sum[m]);
        }
        if constexpr (NM == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[0][j] = silu(sum[0][j]) * sum[1][j];
        }
        if (i < B_real) store4(static_cast<YT*>(a.y) + static_cast<size_t>(i) * a.O + 16 * ob + 4 * q, sum[0], a.accumulate);
    }
}

template <typename XT, typename YT, int NM>
void launch_proj(const ProjArgs& a, hipStream_t s) {
    const int blocks = a.O / 16;
    if (a.B <= 16) {
        proj_stream_kernel<XT, YT, NM, 1, 1, 8><<<dim3(blocks, 1), 8 * kWave, 0, s>>>(a);
    } else {
        proj_stream_kernel<XT, YT, NM, 2, 2, 4>
            <<<dim3((blocks + 1) / 2, (a.B + 31) / 32), 4 * kWave, 0, s>>>(a);
    }
}

template <typename XT>
void launch_shrink(const ProjArgs& a, int tables, hipStream_t s) {
    shrink_kernel<XT><<<dim3((a.B + 15) / 16 * 16, a.max_rank / 16, tables), kShrinkWaves * kWave, 0, s>>>(a);
}

// One projection (NM = 1) or the gate/up pair (NM = 2): shrink, then the product.
template <int NM>
hipError_t run_proj(const ProjArgs& a, hipStream_t s) {
    if (a.adapter != nullptr && a.max_rank > 0 && (a.table[0] != nullptr || (NM == 2 && a.table[1] != nullptr))) {
        if (a.x_dtype == MOE_DT_BF16) launch_shrink<uint16_t>(a, NM, s);
        else launch_shrink<float>(a, NM, s);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.x_dtype == MOE_DT_BF16) {
        if (a.y_dtype == MOE_DT_BF16) launch_proj<uint16_t, uint16_t, NM>(a, s);
        else launch_proj<uint16_t, float, NM>(a, s);
    } else {
        if (a.y_dtype == MOE_DT_BF16) launch_proj<float, uint16_t, NM>(a, s);
        else launch_proj<float, float, NM>(a, s);
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Adapter versions: A [rank, H] into tiles of 16 x 32 and B [O, rank] into
// half tiles of 16 x 16 (lane 16 q + m: row m, ranks 4 q .. 4 q + 3), the rank
// padded to a multiple of 16 with zeros.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void lora_pack_kernel(const uint16_t* __restrict__ src_a,
                                                        const uint16_t* __restrict__ src_b, int rank, int H, int O,
                                                        u32x4* __restrict__ dst_a, u32x2* __restrict__ dst_b) {
    const int nb = (rank + 15) / 16, S = H / 32;
    const long na = static_cast<long>(nb) * S * 64, n_all = na + static_cast<long>(O / 16) * nb * 64;
    for (long c = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; c < n_all;
         c += static_cast<long>(gridDim.x) * blockDim.x) {
        const int lane = static_cast<int>(c & 63), m = lane & 15, q = lane >> 4;
        if (c < na) {
            const long tile = c >> 6;
            const int row = static_cast<int>(tile / S) * 16 + m, col = static_cast<int>(tile % S) * 32 + 8 * q;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (row < rank) v = *reinterpret_cast<const u32x4*>(src_a + static_cast<size_t>(row) * H + col);
            dst_a[c] = v;
        } else {
            const long tile = (c - na) >> 6;
            const size_t row = static_cast<size_t>(tile / nb) * 16 + m;
            const int r0 = static_cast<int>(tile % nb) * 16 + 4 * q;
            uint32_t e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = r0 + j < rank ? src_b[row * rank + r0 + j] : 0u;
            dst_b[c - na] = u32x2{e[0] | (e[1] << 16), e[2] | (e[3] << 16)};
        }
    }
}

__global__ void lora_publish_kernel(moe_lora_handle* table, int i, moe_lora_handle h) {
    if (threadIdx.x == 0) table[i] = h;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t lora_workspace_bytes(int B, int max_rank) {
    return up256(static_cast<size_t>(B) * max_rank * 4);
}

size_t shared_ffn_workspace_bytes(int B, int I, int max_rank, int y_dtype) {
    return 3 * up256(static_cast<size_t>(B) * max_rank * 4) +
           up256(static_cast<size_t>(B) * I * (y_dtype == MOE_DT_F32 ? 4 : 2));
}

hipError_t launch_lora_linear(ProjArgs a, void* ws, hipStream_t s) {
    a.v[0] = static_cast<float*>(ws);
    return run_proj<1>(a, s);
}

hipError_t launch_shared_ffn(ProjArgs a, const void* w_down, const moe_lora_handle* t_down, void* ws, hipStream_t s) {
    char* p = static_cast<char*>(ws);
    const size_t v_bytes = up256(static_cast<size_t>(a.B) * a.max_rank * 4);
    ProjArgs d = a;
    a.v[0] = reinterpret_cast<float*>(p);
    a.v[1] = reinterpret_cast<float*>(p + v_bytes);
    d.v[0] = reinterpret_cast<float*>(p + 2 * v_bytes);
    d.w[0] = w_down;
    d.table[0] = t_down;
    d.table[1] = nullptr;
    d.x = p + 3 * v_bytes;
    d.x_dtype = a.y_dtype;   // h is kept in the output's type
    d.H = a.O;
    d.O = a.H;
    a.y = p + 3 * v_bytes;
    a.accumulate = 0;
    hipError_t e = run_proj<2>(a, s);
    return e != hipSuccess ? e : run_proj<1>(d, s);
}

hipError_t launch_lora_pack(const uint16_t* a, const uint16_t* b, int rank, int H, int O, void* dst_a, void* dst_b,
                            hipStream_t s) {
    const int nb = (rank + 15) / 16;
    const long items = static_cast<long>(nb) * (H / 32) * 64 + static_cast<long>(O / 16) * nb * 64;
    const unsigned grid = static_cast<unsigned>(std::min<long>((items + 255) / 256, 4096));
    lora_pack_kernel<<<grid, 256, 0, s>>>(a, b, rank, H, O, static_cast<u32x4*>(dst_a), static_cast<u32x2*>(dst_b));
    return hipGetLastError();
}

hipError_t launch_lora_publish(moe_lora_handle* table, int i, moe_lora_handle h, hipStream_t s) {
    lora_publish_kernel<<<1, 64, 0, s>>>(table, i, h);
    return hipGetLastError();
}

}  // namespace moe

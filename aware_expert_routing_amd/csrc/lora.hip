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
// c .. c + 7 of its token, as the bf16 terms that enter the product: bf16
// rows (one term), fp32 rows (three, cut in registers) or three bf16 planes
// that hold the cut terms already.
template <int XK>
struct Frag;
template <>
struct Frag<kActBf16> {
    static constexpr int kTerms = 1, kTileBytes = 64, kLaneBytes = 16;
    u32x4 raw;
    __device__ void load(const char* p, size_t) { raw = *reinterpret_cast<const u32x4*>(p); }
    __device__ void terms(u32x4 (&t)[1]) const { t[0] = raw; }
};
template <>
struct Frag<kActF32> {
    static constexpr int kTerms = 3, kTileBytes = 128, kLaneBytes = 32;
    f32x4 lo, hi;
    __device__ void load(const char* p, size_t) {
        lo = *reinterpret_cast<const f32x4*>(p);
        hi = *reinterpret_cast<const f32x4*>(p + 16);
    }
    __device__ void terms(u32x4 (&t)[3]) const {
        const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t s[3][4];
        split<3, 4>(f, s);
#pragma unroll
        for (int i = 0; i < 3; ++i) t[i] = u32x4{s[i][0], s[i][1], s[i][2], s[i][3]};
    }
};
template <>
struct Frag<kActPlanes> {
    static constexpr int kTerms = 3, kTileBytes = 64, kLaneBytes = 16;
    u32x4 raw[3];
    __device__ void load(const char* p, size_t plane) {
#pragma unroll
        for (int i = 0; i < 3; ++i) raw[i] = *reinterpret_cast<const u32x4*>(p + i * plane);
    }
    __device__ void terms(u32x4 (&t)[3]) const {
#pragma unroll
        for (int i = 0; i < 3; ++i) t[i] = raw[i];
    }
};
// Row i of x, the lane's part of it.
template <int XK>
__device__ __forceinline__ const char* x_row(const ProjArgs& a, int i, int q) {
    return static_cast<const char*>(a.x) + static_cast<size_t>(i) * a.H * (Frag<XK>::kTileBytes / 32) +
           q * Frag<XK>::kLaneBytes;
}

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
// shrink: v[i, r] = scale * sum_h A[r, h] x[i, h].  Tokens of one adapter are
// scattered over the batch, so a workgroup gathers its own: it scans the ids
// of a chunk of kChunk tokens, keeps those of its adapter whose place among
// them falls into its part of 16 NT, and multiplies them with RBN rank blocks
// of A; its W waves take the columns' tiles in turn and add their sums in LDS
// in a fixed order.  A workgroup without tokens ends after the scan.
// Workgroups are laid out over the table's entries, or over the chunk's
// tokens (the first token of each adapter stands for it) where those are fewer.
// ---------------------------------------------------------------------------
constexpr int kChunk = 2048;

template <int XK, int NT, int RBN, int W>
__global__ __launch_bounds__(W* kWave) void shrink_kernel(ProjArgs a, int parts, int by_token) {
    __shared__ f32x4 part[W][RBN * NT][kWave];
    __shared__ int tok_s[16 * NT];
    __shared__ int wave_n[W];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int B_real = real_tokens(a);
    const int pieces = (a.max_rank / 16 + RBN - 1) / RBN;   // of rank blocks
    const int t_id = blockIdx.z / pieces, rb0 = (blockIdx.z % pieces) * RBN;
    const int part_id = blockIdx.y % parts, c0 = (blockIdx.y / parts) * kChunk;
    const int c1 = min(c0 + kChunk, B_real);
    const moe_lora_handle* table = a.table[t_id];
    if (table == nullptr || c0 >= c1) return;
    int ad = blockIdx.x;
    if (by_token) {   // this token's adapter, if no earlier token of the chunk has it
        if (c0 + static_cast<int>(blockIdx.x) >= c1) return;
        ad = a.adapter[c0 + blockIdx.x];
        if (ad < 0 || ad >= a.n_adapters) return;
        int dup = 0;
        for (int i = c0 + tid; i < c0 + static_cast<int>(blockIdx.x); i += W * kWave) dup |= a.adapter[i] == ad;
        if (__syncthreads_or(dup)) return;
    }
    const moe_lora_handle h = table[ad];
    const int nb = rank_blocks(h, a.max_rank);
    if (rb0 >= nb) return;

    // the chunk's tokens of this adapter, in order: places part_id 16 NT ..
    if (tid < 16 * NT) tok_s[tid] = -1;
    int base = -part_id * 16 * NT;   // place of the next match, relative to this part
    for (int i0 = c0; i0 < c1; i0 += W * kWave) {
        const int i = i0 + tid;
        const bool m = i < c1 && a.adapter[i] == ad;
        const uint64_t b = __ballot(m);
        if (lane == 0) wave_n[wave] = __popcll(b);
        __syncthreads();
        int at = base + __popcll(b & ((1ull << lane) - 1ull));
#pragma unroll
        for (int w = 0; w < W; ++w) {
            at += w < wave ? wave_n[w] : 0;
            base += wave_n[w];
        }
        if (m && at >= 0 && at < 16 * NT) tok_s[at] = i;
        __syncthreads();
        if (base >= 16 * NT) break;
    }
    const int have = min(base, 16 * NT);
    if (have <= 0) return;

    const int S = a.H / 32;
    const char* A[RBN];
#pragma unroll
    for (int r = 0; r < RBN; ++r)
        A[r] = static_cast<const char*>(h.a) + static_cast<size_t>(min(rb0 + r, nb - 1)) * S * 1024 + lane * 16;
    const char* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = x_row<XK>(a, tok_s[min(16 * t + n, have - 1)], q);
    f32x4 acc[RBN][NT];
#pragma unroll
    for (int r = 0; r < RBN; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kU = (RBN + NT) * (Frag<XK>::kTerms > 1 ? 2 : 1) > 4 ? 2 : 4;
    const int nt = (have + 15) / 16;
#pragma unroll kU
    for (int s = wave; s < S; s += W) {
        u32x4 w[RBN];
#pragma unroll
        for (int r = 0; r < RBN; ++r) w[r] = *reinterpret_cast<const u32x4*>(A[r] + static_cast<size_t>(s) * 1024);
        Frag<XK> f[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t < nt) f[t].load(xp[t] + static_cast<size_t>(s) * Frag<XK>::kTileBytes, a.x_plane);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
            u32x4 x[Frag<XK>::kTerms];
            f[t].terms(x);
#pragma unroll
            for (int k = Frag<XK>::kTerms - 1; k >= 0; --k)
#pragma unroll
                for (int r = 0; r < RBN; ++r) acc[r][t] = mma32(w[r], x[k], acc[r][t]);
        }
    }
#pragma unroll
    for (int r = 0; r < RBN; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][r * NT + t][lane] = acc[r][t];
    __syncthreads();
    for (int p = wave; p < RBN * NT; p += W) {
        const int r = p / NT, t = p % NT;
        if (rb0 + r >= nb || 16 * t + n >= have) continue;
        f32x4 v = part[0][p][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][p][lane];
        float* out = a.v[t_id] + static_cast<size_t>(tok_s[16 * t + n]) * a.max_rank + 16 * (rb0 + r) + 4 * q;
        *reinterpret_cast<f32x4*>(out) = v * h.scale;
    }
}

// Rank block r of the lane's token's v as bf16 terms (zero where !mine).
template <int VT>
__device__ __forceinline__ void v_terms(const float* v_row, int r, int q, bool mine, u32x2 (&out)[VT]) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mine) v = *reinterpret_cast<const f32x4*>(v_row + 16 * r + 4 * q);
    const float f[4] = {v.x, v.y, v.z, v.w};
    uint32_t t[VT][2];
    split<VT, 2>(f, t);
#pragma unroll
    for (int k = 0; k < VT; ++k) out[k] = u32x2{t[k][0], t[k][1]};
}

// Adds B_a v to the accumulators of MB row blocks and NB tiles of 16 tokens
// (i0 the first token), one adapter of those tokens after the other.  Of
// adapter d's rank blocks r those with (d + r) mod step == first (step a power
// of two): which wave adds a token's part does not depend on the other
// tokens.  ob(j): row block of accumulator row j, mat(j): its matrix.
template <int VT, int MB, int NB, typename Ob, typename Mat>
__device__ __forceinline__ void expand(const ProjArgs& a, int i0, int B_real, int first, int step,
                                       f32x4 (&acc)[MB][NB], Ob ob, Mat mat) {
    static_assert(NB <= 4, "a token per lane");
    if (a.adapter == nullptr) return;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, q = lane >> 4;
    const int id = lane < 16 * NB ? adapter_of(a, i0 + lane, B_real) : -1;   // lane = token
    uint64_t rem = __ballot(id >= 0);
    while (rem != 0ull) {
        const int ad = __builtin_amdgcn_readlane(id, __ffsll(static_cast<unsigned long long>(rem)) - 1);
        const uint64_t who = __ballot(id == ad);
        rem &= ~who;
        constexpr bool kTwo = MB > 1;
        moe_lora_handle h[2];
        int nb[2] = {0, 0};
#pragma unroll
        for (int m = 0; m < (kTwo ? 2 : 1); ++m)
            if (a.table[m] != nullptr) {
                h[m] = a.table[m][ad];
                nb[m] = rank_blocks(h[m], a.max_rank);
            }
        const int most = max(nb[0], nb[1]);
        for (int r = (first - ad) & (step - 1); r < most; r += step) {
            u32x2 b[MB];
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                const int m = mat(j);
                b[j] = u32x2{0u, 0u};
                if (r < nb[m])
                    b[j] = *reinterpret_cast<const u32x2*>(static_cast<const char*>(h[m].b) +
                                                           (static_cast<size_t>(ob(j)) * nb[m] + r) * 512 + lane * 8);
            }
#pragma unroll
            for (int t = 0; t < NB; ++t) {
                if (((who >> (16 * t)) & 0xffffull) == 0ull) continue;
                const bool mine = (who >> (16 * t + n)) & 1ull;
                const size_t row = static_cast<size_t>(min(i0 + 16 * t + n, B_real - 1)) * a.max_rank;
#pragma unroll
                for (int m = 0; m < (kTwo ? 2 : 1); ++m) {
                    if (r >= nb[m]) continue;
                    u32x2 v[VT];
                    v_terms<VT>(a.v[m] + row, r, q, mine, v);
#pragma unroll
                    for (int j = 0; j < MB; ++j) {
                        if (mat(j) != m) continue;
#pragma unroll
                        for (int k = VT - 1; k >= 0; --k) acc[j][t] = mma16(b[j], v[k], acc[j][t]);
                    }
                }
            }
        }
    }
}

__device__ __forceinline__ float silu(float z) { return z / (1.0f + __expf(-z)); }

// Four consecutive outputs (columns c .. c + 3) of token i.
template <int YK>
__device__ __forceinline__ void store4(const ProjArgs& a, int i, int c, f32x4 v) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const size_t at = static_cast<size_t>(i) * a.O + c;
    if constexpr (YK == kActF32) {
        float* p = static_cast<float*>(a.y) + at;
        if (a.accumulate) v += *reinterpret_cast<const f32x4*>(p);
        *reinterpret_cast<f32x4*>(p) = v;
    } else if constexpr (YK == kActBf16) {
        *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) =
            __builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4));
    } else {
        const float f[4] = {v.x, v.y, v.z, v.w};
        uint32_t t[3][2];
        split<3, 2>(f, t);
#pragma unroll
        for (int k = 0; k < 3; ++k)
            *reinterpret_cast<u32x2*>(static_cast<char*>(a.y) + k * a.y_plane + at * 2) = u32x2{t[k][0], t[k][1]};
    }
}
template <int YK>
constexpr int v_terms_for() { return YK == kActBf16 ? 2 : 3; }

// ---------------------------------------------------------------------------
// Streaming projection, for few tokens: a workgroup owns RB row blocks of 16
// outputs (of NM matrices: 2 = gate and up, whose result is silu(g) u) and NT
// tiles of 16 tokens.  Its W waves take the columns' tiles in turn, and the
// adapters of the tokens in turn, and add their sums in LDS in a fixed order.
// ---------------------------------------------------------------------------
template <int XK, int YK, int NM, int NT, int RB, int W, int U>
__global__ __launch_bounds__(W* kWave) void proj_stream_kernel(ProjArgs a) {
    constexpr int TT = Frag<XK>::kTerms;
    constexpr int MB = NM * RB;
    __shared__ f32x4 part[W][MB * NT][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int B_real = real_tokens(a);
    const int i0 = blockIdx.y * 16 * NT;
    if (i0 >= B_real) return;
    const int ob0 = blockIdx.x * RB, blocks = a.O / 16;
    const int S = a.H / 32;

    const char* wp[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j)
        wp[j] = static_cast<const char*>(a.w[j / RB]) +
                static_cast<size_t>(min(ob0 + j % RB, blocks - 1)) * S * 1024 + lane * 16;
    const char* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = x_row<XK>(a, min(i0 + 16 * t + n, B_real - 1), q);

    f32x4 acc[MB][NT];
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[j][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll U
    for (int s = wave; s < S; s += W) {
        u32x4 w[MB];
        Frag<XK> f[NT];
#pragma unroll
        for (int j = 0; j < MB; ++j) w[j] = *reinterpret_cast<const u32x4*>(wp[j] + static_cast<size_t>(s) * 1024);
#pragma unroll
        for (int t = 0; t < NT; ++t) f[t].load(xp[t] + static_cast<size_t>(s) * Frag<XK>::kTileBytes, a.x_plane);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            u32x4 x[TT];
            f[t].terms(x);
#pragma unroll
            for (int k = TT - 1; k >= 0; --k)
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[j][t] = mma32(w[j], x[k], acc[j][t]);
        }
    }
    expand<v_terms_for<YK>()>(a, i0, B_real, wave, W, acc, [&](int j) { return min(ob0 + j % RB, blocks - 1); },
                              [&](int j) { return j / RB; });
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][j * NT + t][lane] = acc[j][t];
    __syncthreads();
    for (int p = wave; p < RB * NT; p += W) {
        const int r = p / NT, t = p % NT;
        const int ob = ob0 + r, i = i0 + 16 * t + n;
        if (ob >= blocks || i >= B_real) continue;
        f32x4 sum[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            sum[m] = part[0][m * RB * NT + p][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum[m] += part[w][m * RB * NT + p][lane];
        }
        if constexpr (NM == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[0][j] = silu(sum[0][j]) * sum[1][j];
        }
        store4<YK>(a, i, 16 * ob + 4 * q, sum[0]);
    }
}

// ---------------------------------------------------------------------------
// Tiled projection, for many tokens: a workgroup of WR x WC waves owns
// 16 WR MB rows of W (for NM = 2 half of them gate rows and half the up rows of
// the same outputs) and 16 WC NB tokens; a wave owns MB x NB blocks of 16 x 16
// in accumulators.  Two column tiles at a time are copied to LDS in operand
// order (a packed weight tile as it lies; of x the lane's 16 bytes of its
// token's row), straight from memory (global_load_lds), into the half of a
// double buffer that the products are not reading.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(1))) const void* gptr;
typedef __attribute__((address_space(3))) void* lptr;

template <int XK, int YK, int NM, int WR, int WC, int MB, int NB>
__global__ __launch_bounds__(WR* WC* kWave) void proj_tile_kernel(ProjArgs a, int row_tiles, int tok_tiles) {
    constexpr int NW = WR * WC;
    constexpr int RT = WR * MB, CT = WC * NB;      // 1 KB tiles per 32 columns
    constexpr int kStep = RT + CT;
    constexpr int kStage = 2 * kStep * 1024;
    constexpr int kPer = 2 * kStep / NW;           // tiles a wave copies per stage
    static_assert(2 * kStep % NW == 0 && MB % NM == 0, "tile split");
    constexpr int P = XK == kActPlanes ? 3 : 1;
    __shared__ __align__(1024) char lds[2 * kStage];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int wr = wave / WC, wc = wave % WC;
    const int B_real = real_tokens(a);
    const int tile_r = blockIdx.x % row_tiles, tile_c = blockIdx.x / row_tiles;
    const int i0 = tile_c * 16 * CT;
    if (i0 >= B_real) return;
    const int blocks = a.O / 16, S = a.H / 32, steps = P * S;
    const int ob0 = tile_r * (RT / NM);
    // output row block and matrix of row tile j of the workgroup
    constexpr int kHalf = MB / NM;
    auto mat_of = [](int j) { return NM == 1 ? 0 : (j % MB) / kHalf; };
    auto ob_of = [&](int j) { return min(ob0 + (NM == 1 ? j : (j / MB) * kHalf + j % kHalf), blocks - 1); };

    const char* src[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int slot = wave * kPer + u, j = slot >> 1;
        if (j < RT)
            src[u] = static_cast<const char*>(mat_of(j) ? a.w[1] : a.w[0]) + static_cast<size_t>(ob_of(j)) * S * 1024 +
                     lane * 16;
        else
            src[u] = x_row<kActBf16>(a, min(i0 + 16 * (j - RT) + n, B_real - 1), q);
    }
    auto copy = [&](int it, int buf) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int slot = wave * kPer + u, j = slot >> 1;
            const int kk = min(2 * it + (slot & 1), steps - 1);
            const int plane = P == 1 ? 0 : P - 1 - kk / S;   // the smallest term first
            const int s = P == 1 ? kk : kk % S;
            const char* g = src[u] + (j < RT ? static_cast<size_t>(s) * 1024
                                             : static_cast<size_t>(s) * 64 + static_cast<size_t>(plane) * a.x_plane);
            __builtin_amdgcn_global_load_lds((gptr)g, (lptr)(lds + buf * kStage + ((slot & 1) * kStep + j) * 1024), 16,
                                             0, 0);
        }
    };

    f32x4 acc[MB][NB];
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int t = 0; t < NB; ++t) acc[j][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    copy(0, 0);
    __syncthreads();
    auto multiply = [&](int buf, int ks) {
        const char* base = lds + buf * kStage + ks * kStep * 1024 + lane * 16;
        u32x4 w[MB], x[NB];
#pragma unroll
        for (int t = 0; t < NB; ++t) x[t] = *reinterpret_cast<const u32x4*>(base + (RT + wc * NB + t) * 1024);
#pragma unroll
        for (int j = 0; j < MB; ++j) w[j] = *reinterpret_cast<const u32x4*>(base + (wr * MB + j) * 1024);
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int t = 0; t < NB; ++t) acc[j][t] = mma32(w[j], x[t], acc[j][t]);
    };
    const int its = (steps + 1) / 2;
    for (int it = 0; it + 1 < its; ++it) {
        copy(it + 1, (it & 1) ^ 1);
        multiply(it & 1, 0);
        multiply(it & 1, 1);
        __syncthreads();
    }
    multiply((its - 1) & 1, 0);
    if ((steps & 1) == 0) multiply((its - 1) & 1, 1);
    expand<v_terms_for<YK>()>(a, i0 + 16 * NB * wc, B_real, 0, 1, acc,
                              [&](int j) { return ob_of(wr * MB + j); }, [&](int j) { return mat_of(j); });
#pragma unroll
    for (int j = 0; j < kHalf; ++j) {
        const int ob = ob0 + wr * kHalf + j;
        if (ob >= blocks) continue;
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const int i = i0 + 16 * (NB * wc + t) + n;
            f32x4 r = acc[j][t];
            if constexpr (NM == 2) {
#pragma unroll
                for (int e = 0; e < 4; ++e) r[e] = silu(r[e]) * acc[j + kHalf][t][e];
            }
            if (i < B_real) store4<YK>(a, i, 16 * ob + 4 * q, r);
        }
    }
}

// fp32 rows cut into their three bf16 terms, as planes.
__global__ __launch_bounds__(256) void planes_kernel(const f32x4* __restrict__ x, long chunks, u32x2* __restrict__ out,
                                                     size_t plane) {
    for (long c = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; c < chunks;
         c += static_cast<long>(gridDim.x) * blockDim.x) {
        const f32x4 v = x[c];
        const float f[4] = {v.x, v.y, v.z, v.w};
        uint32_t t[3][2];
        split<3, 2>(f, t);
#pragma unroll
        for (int k = 0; k < 3; ++k) out[k * plane / 8 + c] = u32x2{t[k][0], t[k][1]};
    }
}

constexpr int kStreamTokens = 128;   // up to this many: the streaming kernel
constexpr int kRowTokens = 16;       // up to this many: fp32 rows are cut in registers

template <int XK, int YK, int NM, int NT, int W, int U>
void launch_stream(const ProjArgs& a, hipStream_t s) {
    proj_stream_kernel<XK, YK, NM, NT, 1, W, U>
        <<<dim3(a.O / 16, (a.B + 16 * NT - 1) / (16 * NT)), W * kWave, 0, s>>>(a);
}
template <int XK, int YK, int NM, int WR, int WC, int MB, int NB>
hipError_t launch_tile(const ProjArgs& a, hipStream_t s) {
    constexpr int kRows = 16 * WR * MB / NM, kTok = 16 * WC * NB;
    const int rt = (a.O + kRows - 1) / kRows, ct = (a.B + kTok - 1) / kTok;
    proj_tile_kernel<XK, YK, NM, WR, WC, MB, NB><<<static_cast<unsigned>(rt) * ct, WR * WC * kWave, 0, s>>>(a, rt, ct);
    return hipGetLastError();
}

template <int XK, int YK, int NM>
hipError_t launch_proj(const ProjArgs& a, hipStream_t s) {
    if (a.B <= 16) launch_stream<XK, YK, NM, 1, 8, 4>(a, s);
    else if constexpr (XK != kActF32) {
        if (a.B <= 32) launch_stream<XK, YK, NM, 2, 8, 4>(a, s);
        else if (a.B <= kStreamTokens) launch_stream<XK, YK, NM, 4, 8 / NM, 2>(a, s);
        else {
            const long big = (static_cast<long>(a.O) * NM + 255) / 256 * ((a.B + 255) / 256);
            return big >= 128 ? launch_tile<XK, YK, NM, 2, 4, 8, 4>(a, s) : launch_tile<XK, YK, NM, 2, 2, 4, 4>(a, s);
        }
    }
    return hipGetLastError();
}

template <int XK, int NT, int RBN, int W>
void launch_shrink_as(const ProjArgs& a, int tables, hipStream_t s) {
    const int chunk = std::min(a.B, kChunk), chunks = (a.B + kChunk - 1) / kChunk;
    const int parts = (chunk + 16 * NT - 1) / (16 * NT);
    const int by_token = a.n_adapters > chunk;
    const int pieces = (a.max_rank / 16 + RBN - 1) / RBN;
    shrink_kernel<XK, NT, RBN, W><<<dim3(by_token ? chunk : a.n_adapters, parts * chunks, pieces * tables), W * kWave, 0,
                                    s>>>(a, parts, by_token);
}
template <int XK>
void launch_shrink(const ProjArgs& a, int tables, hipStream_t s) {
    if (a.B <= 128) launch_shrink_as<XK, 1, 1, 8>(a, tables, s);
    else launch_shrink_as<XK, 4, 2, 8>(a, tables, s);
}

// One projection (NM = 1) or the gate/up pair (NM = 2): shrink, then the product.
template <int NM>
hipError_t run_proj(const ProjArgs& a, hipStream_t s) {
    if (a.adapter != nullptr && (a.table[0] != nullptr || (NM == 2 && a.table[1] != nullptr))) {
        if (a.x_kind == kActBf16) launch_shrink<kActBf16>(a, NM, s);
        else if (a.x_kind == kActPlanes) launch_shrink<kActPlanes>(a, NM, s);
        else launch_shrink<kActF32>(a, NM, s);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
#define MOE_PROJ(X_, Y_) \
    if (a.x_kind == X_ && a.y_kind == Y_) return launch_proj<X_, Y_, NM>(a, s)
    MOE_PROJ(kActBf16, kActBf16);
    MOE_PROJ(kActF32, kActBf16);
    MOE_PROJ(kActPlanes, kActBf16);
    if constexpr (NM == 1) {
        MOE_PROJ(kActBf16, kActF32);
        MOE_PROJ(kActF32, kActF32);
        MOE_PROJ(kActPlanes, kActF32);
    } else {
        MOE_PROJ(kActBf16, kActPlanes);
        MOE_PROJ(kActF32, kActPlanes);
        MOE_PROJ(kActPlanes, kActPlanes);
    }
#undef MOE_PROJ
    return hipErrorInvalidValue;
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
size_t v_bytes(int B, int max_rank) { return up256(static_cast<size_t>(B) * max_rank * 4); }
size_t x_planes_bytes(int B, int H, int x_dtype) {   // fp32 x of more than kRowTokens tokens
    return x_dtype == MOE_DT_F32 && B > kRowTokens ? 3 * up256(static_cast<size_t>(B) * H * 2) : 0;
}

// Cut an fp32 x into planes at `ws` where the call's kernels read planes.
hipError_t cut_x(ProjArgs& a, void* ws, hipStream_t s) {
    if (a.x_kind != kActF32 || a.B <= kRowTokens) return hipSuccess;
    const size_t plane = up256(static_cast<size_t>(a.B) * a.H * 2);
    const long chunks = static_cast<long>(a.B) * a.H / 4;
    planes_kernel<<<static_cast<unsigned>(std::min<long>((chunks + 255) / 256, 4096)), 256, 0, s>>>(
        static_cast<const f32x4*>(a.x), chunks, static_cast<u32x2*>(ws), plane);
    a.x = ws;
    a.x_kind = kActPlanes;
    a.x_plane = plane;
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int B, int H, int max_rank, int x_dtype) {
    return v_bytes(B, max_rank) + x_planes_bytes(B, H, x_dtype);
}

// v of gate, up and down, the planes of x, h (bf16, or three planes for an fp32 y).
size_t shared_ffn_workspace_bytes(int B, int H, int I, int max_rank, int x_dtype, int y_dtype) {
    return 3 * v_bytes(B, max_rank) + x_planes_bytes(B, H, x_dtype) +
           (y_dtype == MOE_DT_F32 ? 3 : 1) * up256(static_cast<size_t>(B) * I * 2);
}

hipError_t launch_lora_linear(ProjArgs a, void* ws, hipStream_t s) {
    a.v[0] = static_cast<float*>(ws);
    hipError_t e = cut_x(a, static_cast<char*>(ws) + v_bytes(a.B, a.max_rank), s);
    return e != hipSuccess ? e : run_proj<1>(a, s);
}

hipError_t launch_shared_ffn(ProjArgs a, const void* w_down, const moe_lora_handle* t_down, void* ws, hipStream_t s) {
    char* p = static_cast<char*>(ws);
    const size_t vb = v_bytes(a.B, a.max_rank);
    const size_t h_plane = up256(static_cast<size_t>(a.B) * a.O * 2);
    ProjArgs d = a;
    a.v[0] = reinterpret_cast<float*>(p);
    a.v[1] = reinterpret_cast<float*>(p + vb);
    d.v[0] = reinterpret_cast<float*>(p + 2 * vb);
    char* x_planes = p + 3 * vb;
    char* h = x_planes + x_planes_bytes(a.B, a.H, a.x_kind == kActF32 ? MOE_DT_F32 : MOE_DT_BF16);
    a.y = h;
    a.y_kind = a.y_kind == kActF32 ? kActPlanes : kActBf16;
    a.y_plane = h_plane;
    a.accumulate = 0;
    d.w[0] = w_down;
    d.table[0] = t_down;
    d.table[1] = nullptr;
    d.x = h;
    d.x_kind = a.y_kind;
    d.x_plane = h_plane;
    d.H = a.O;
    d.O = a.H;
    hipError_t e = cut_x(a, x_planes, s);
    if (e == hipSuccess) e = run_proj<2>(a, s);
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

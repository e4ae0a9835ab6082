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
// v_i = s_a A_a x_i is formed in fp32 first, and B_a v_i is added before the
// outputs are stored.  By sizes (plan_proj):
//   few tokens with few rank blocks   one launch (proj_fused_kernel)
//   a decode batch                    the product split over its columns, beside
//                                     it v and the lists of adapters, in one
//                                     launch (proj_split_kernel); the sums, B v
//                                     and the epilogue in a second one
//                                     (proj_finish_kernel)
//   many tokens                       v (shrink_kernel), then a tiled product
//                                     that adds B v behind its columns
//                                     (proj_tile_kernel)
// Few tokens are bound by latency and by what one compute unit can have in
// flight, a decode batch by the weights' way from memory and the two launches,
// many tokens by the matrix units.  Measured on an MI355X, kernel time, with
// adapters: 1 token of 2048 x 2048 5.7 us (weights alone at the copy rate of
// 4.8 TB/s: 1.8); 64 tokens of 4096 x 4096 with 24 adapters 21 us (9.7); 4096
// tokens of 4096 x 4096 with 8 adapters 134 us, without 117, where the matrix
// units' rate in a large library product (1.40 PFLOP/s) gives 98.  The shared
// expert: 1 token of H = 2048, I = 768 with an adapter 13 us (2.0), 128 of 4096,
// 1536 with 24 adapters 60 (15), 2999 of the same with 6 adapters 175 alone and
// 152 where calls follow each other (82).
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
// infinity, whose difference to itself is NaN; a NaN stays one, also where its
// set bits all lie in the lower half).
__device__ __forceinline__ float cut8(float f, float& rest) {
    const float t = __uint_as_float(__float_as_uint(f) & 0xffff0000u);
    const float r = f - t;
    rest = r == r ? r : 0.0f;
    return f == f ? t : __uint_as_float(0x7fc00000u);
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
// The fragments of a pair of column tiles for NT tiles of 16 tokens, loaded as
// whole lines: a fragment takes 16 bytes from each of 16 rows, and a load that
// does so touches eight times the cache lines of one in which eight lanes take
// a row's 128 bytes.  Lane l loads chunk l % 8 of row 8 h + l / 8; the wave turns
// that into fragments through 2 KB of LDS per tile that it alone uses (LDS
// operations of a wave stay in order, so nothing is waited for but the data).
// Chunk c of row r lies at place c ^ (r / 2 mod 8), so that 16 rows' chunks lie
// in different banks.  bf16 rows and planes; fp32 rows are read as fragments.
template <int XK, int NT>
struct Lines {
    static constexpr int kParts = XK == kActPlanes ? 3 : 1;
    u32x4 v[NT][2][kParts];
    // rows: byte offsets of the lane's rows from x
    __device__ __forceinline__ void load(const ProjArgs& a, const uint32_t (&rows)[NT][2], int pair) {
        const char* x = static_cast<const char*>(a.x) + static_cast<size_t>(pair) * 128;
#pragma unroll
        for (int k = 0; k < kParts; ++k)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[t][h][k] = *reinterpret_cast<const u32x4*>(x + k * a.x_plane + rows[t][h]);
    }
    // Part k's fragments of both column tiles: frag[h][t].
    __device__ __forceinline__ void turn(char* lds, int k, u32x4 (&frag)[2][NT]) const {
        const int lane = threadIdx.x & (kWave - 1), n = lane & 15, q = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 8 * h + (lane >> 3);
                *reinterpret_cast<u32x4*>(lds + t * 2048 + r * 128 + (((lane & 7) ^ ((r >> 1) & 7)) * 16)) = v[t][h][k];
            }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                frag[h][t] = *reinterpret_cast<const u32x4*>(lds + t * 2048 + n * 128 +
                                                             (((4 * h + q) ^ ((n >> 1) & 7)) * 16));
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
// of a chunk of tokens [c0, c1), keeps those of its adapter whose place among
// them falls into a part of 16 NT, and multiplies them with RBN rank blocks
// of A; its W waves take pairs of the columns' tiles in turn (a pair is one
// 128-byte line of a bf16 row) and add their sums in LDS in a fixed order.
// ---------------------------------------------------------------------------
constexpr int kChunk = 2048;

template <int NT, int RBN, int W>
struct ShrinkLds {
    union {
        f32x4 part[W / 2][RBN * NT][kWave];
        char lines[W][NT * 2048];
    };
    int tok[16 * NT];
    int found[kChunk / kWave];
};

// Adds the W waves' accumulator blocks (T of them, in order wave, wave + W/2)
// pairwise into part[0 .. W/2 - 1]; the caller's threads are synchronised after.
template <int W, int T>
__device__ __forceinline__ void fold_waves(f32x4 (*part)[T][kWave], const f32x4 (&acc)[T], int wave, int lane) {
    if (wave >= W / 2)
#pragma unroll
        for (int p = 0; p < T; ++p) part[wave - W / 2][p][lane] = acc[p];
    __syncthreads();
    if (wave < W / 2)
#pragma unroll
        for (int p = 0; p < T; ++p) part[wave][p][lane] = acc[p] + part[wave][p][lane];
    __syncthreads();
}

// Parts first_part, first_part + step, .. of adapter ad's tokens, rank blocks
// rb0 .. of table t_id; c1 - c0 <= kChunk.
template <int XK, int NT, int RBN, int W>
__device__ __forceinline__ void shrink_block(const ProjArgs& a, ShrinkLds<NT, RBN, W>& l, int t_id, int ad, int rb0,
                                             int c0, int c1, int first_part, int step) {
    constexpr int U = kChunk / (W * kWave);   // ids a thread looks at
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int n = lane & 15, q = lane >> 4;
    const moe_lora_handle h = a.table[t_id][ad];
    const int nb = rank_blocks(h, a.max_rank);
    if (rb0 >= nb) return;
    // the chunk's tokens of this adapter: their number, and this thread's places among them
    int at[U];
    uint64_t b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = c0 + u * W * kWave + tid;
        b[u] = __ballot(i < c1 && a.adapter[i] == ad);
        if (lane == 0) l.found[u * W + wave] = __popcll(b[u]);
    }
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = all + __popcll(b[u] & ((1ull << lane) - 1ull));
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int f = l.found[u * W + w];
            at[u] += w < wave ? f : 0;
            all += f;
        }
    }
    const int S = a.H / 32;
    const char* A[RBN];
#pragma unroll
    for (int r = 0; r < RBN; ++r)
        A[r] = static_cast<const char*>(h.a) + static_cast<size_t>(min(rb0 + r, nb - 1)) * S * 1024 + lane * 16;
    for (int base = first_part * 16 * NT; base < all; base += step * 16 * NT) {
        const int have = min(all - base, 16 * NT);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (((b[u] >> lane) & 1ull) && at[u] >= base && at[u] < base + 16 * NT)
                l.tok[at[u] - base] = c0 + u * W * kWave + tid;
        __syncthreads();
        const char* xp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xp[t] = x_row<XK>(a, l.tok[min(16 * t + n, have - 1)], q);
        f32x4 acc[RBN * NT];
#pragma unroll
        for (int p = 0; p < RBN * NT; ++p) acc[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        auto tile = [&](int s) {
            u32x4 w[RBN];
#pragma unroll
            for (int r = 0; r < RBN; ++r) w[r] = *reinterpret_cast<const u32x4*>(A[r] + static_cast<size_t>(s) * 1024);
            Frag<XK> f[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) f[t].load(xp[t] + static_cast<size_t>(s) * Frag<XK>::kTileBytes, a.x_plane);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                u32x4 x[Frag<XK>::kTerms];
                f[t].terms(x);
#pragma unroll
                for (int k = Frag<XK>::kTerms - 1; k >= 0; --k)
#pragma unroll
                    for (int r = 0; r < RBN; ++r) acc[r * NT + t] = mma32(w[r], x[k], acc[r * NT + t]);
            }
        };
        // kU pairs of a wave in flight: about 24 loads
        constexpr int kLoads = 2 * (RBN + NT * (XK == kActF32 ? 2 : Frag<XK>::kTerms));
        constexpr int kU = kLoads >= 12 ? 1 : (kLoads > 6 ? 2 : 4);
        const int pairs = S / 2;
        if constexpr (XK == kActF32) {
#pragma unroll kU
            for (int s = wave; s < pairs; s += W) {
                tile(2 * s);
                tile(2 * s + 1);
            }
        } else {
            uint32_t rows[NT][2];   // from the chunk's first token
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    rows[t][k] = static_cast<uint32_t>(l.tok[min(16 * t + 8 * k + (lane >> 3), have - 1)] - c0) *
                                     (a.H * 2) + (lane & 7) * 16;
            ProjArgs c = a;
            c.x = static_cast<const char*>(a.x) + static_cast<size_t>(c0) * a.H * 2;
            for (int s = wave; s < pairs; s += W * kU) {
                u32x4 w[kU][2][RBN];
                Lines<XK, NT> x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int p = s + u * W;
                    if (p >= pairs) continue;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int r = 0; r < RBN; ++r)
                            w[u][k][r] = *reinterpret_cast<const u32x4*>(A[r] + static_cast<size_t>(2 * p + k) * 1024);
                    x[u].load(c, rows, p);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (s + u * W >= pairs) continue;
#pragma unroll
                    for (int k = Lines<XK, NT>::kParts - 1; k >= 0; --k) {
                        u32x4 f[2][NT];
                        x[u].turn(l.lines[wave], k, f);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < RBN; ++r)
#pragma unroll
                                for (int g = 0; g < 2; ++g)
                                    acc[r * NT + t] = mma32(w[u][g][r], f[g][t], acc[r * NT + t]);
                    }
                }
            }
        }
        if ((S & 1) && wave == W - 1) tile(S - 1);
        __syncthreads();   // the lines' room becomes the sums'
        fold_waves<W>(l.part, acc, wave, lane);
        for (int p = wave; p < RBN * NT; p += W) {
            const int r = p / NT, t = p % NT;
            if (rb0 + r >= nb || 16 * t + n >= have) continue;
            f32x4 v = l.part[0][p][lane];
#pragma unroll
            for (int w = 1; w < W / 2; ++w) v += l.part[w][p][lane];
            float* out = a.v[t_id] + static_cast<size_t>(l.tok[16 * t + n]) * a.max_rank + 16 * (rb0 + r) + 4 * q;
            *reinterpret_cast<f32x4*>(out) = v * h.scale;
        }
        __syncthreads();
    }
}

// Workgroups of a chunk are laid out over the table's entries, or over the
// chunk's tokens (the first token of each adapter stands for it) where those
// are fewer.  The adapter of place `at`, -1: none here.  Uniform over the
// workgroup; every thread calls it.
__device__ __forceinline__ int shrink_adapter(const ProjArgs& a, int at, int by_token, int c0, int c1) {
    if (!by_token) return at;
    if (c0 + at >= c1) return -1;
    const int ad = a.adapter[c0 + at];
    if (ad < 0 || ad >= a.n_adapters) return -1;
    int dup = 0;
    for (int i = c0 + static_cast<int>(threadIdx.x); i < c0 + at; i += blockDim.x) dup |= a.adapter[i] == ad;
    return __syncthreads_or(dup) ? -1 : ad;
}

// grid: (places, parts x chunks, pieces of rank blocks x tables)
template <int XK, int NT, int RBN, int W>
__global__ __launch_bounds__(W* kWave) void shrink_kernel(ProjArgs a, int parts, int by_token) {
    __shared__ ShrinkLds<NT, RBN, W> l;
    const int pieces = (a.max_rank / 16 + RBN - 1) / RBN;
    const int t_id = blockIdx.z / pieces, rb0 = (blockIdx.z % pieces) * RBN;
    const int c0 = (blockIdx.y / parts) * kChunk, c1 = min(c0 + kChunk, real_tokens(a));
    if (a.table[t_id] == nullptr || c0 >= c1) return;
    const int ad = shrink_adapter(a, blockIdx.x, by_token, c0, c1);
    if (ad >= 0) shrink_block<XK, NT, RBN, W>(a, l, t_id, ad, rb0, c0, c1, blockIdx.y % parts, parts);
}

__device__ __forceinline__ uint32_t lane_u32(uint32_t v, int l) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l));
}

// Adds B_a v to the accumulators of MB row blocks (of NM matrices) and 64
// tokens (i0 the first), one rank block of one adapter after the other; the
// next one's operands are loaded before the present one's products.  ob(j):
// row block of accumulator row j, mat(j): its matrix.
template <int VT, int NM, int MB, typename Ob, typename Mat>
__device__ __forceinline__ void expand(const ProjArgs& a, int i0, int B_real, f32x4 (&acc)[MB][4], Ob ob, Mat mat) {
    if (a.adapter == nullptr) return;
    const int lane = threadIdx.x & (kWave - 1), n = lane & 15, q = lane >> 4;
    const int id = adapter_of(a, i0 + lane, B_real);   // lane = token
    // every lane reads its own token's handles, all of them in one round trip
    int nb[NM];
    uint64_t hb[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        nb[m] = 0;
        hb[m] = 0;
        if (a.table[m] != nullptr && id >= 0) {
            const moe_lora_handle* h = a.table[m] + id;
            nb[m] = rank_blocks(*h, a.max_rank);
            hb[m] = reinterpret_cast<uint64_t>(h->b);
        }
    }
    bool any = nb[0] > 0;
    if constexpr (NM == 2) any = any || nb[1] > 0;
    uint64_t rem = __ballot(any);
    struct Item {
        uint64_t who;
        const char* b[NM];
        int nb[NM], r;
    } cur{}, nxt{};
    nxt.r = -1;
    auto next = [&](Item& it) {   // the rank block after `it`, false: none
        int most = it.nb[0];
        if constexpr (NM == 2) most = max(most, it.nb[1]);
        if (++it.r < most) return true;
        if (rem == 0ull) return false;
        const int from = __ffsll(static_cast<unsigned long long>(rem)) - 1;
        const int ad = __builtin_amdgcn_readlane(id, from);
        it.who = __ballot(id == ad);
        rem &= ~it.who;
        it.r = 0;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            it.nb[m] = __builtin_amdgcn_readlane(nb[m], from);
            it.b[m] = reinterpret_cast<const char*>(
                (static_cast<uint64_t>(lane_u32(static_cast<uint32_t>(hb[m] >> 32), from)) << 32) |
                lane_u32(static_cast<uint32_t>(hb[m]), from));
        }
        return true;
    };
    auto load = [&](const Item& it, u32x2 (&b)[MB], f32x4 (&v)[NM][4]) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int m = mat(j);
            b[j] = u32x2{0u, 0u};
            if (it.r < it.nb[m])
                b[j] = *reinterpret_cast<const u32x2*>(it.b[m] + (static_cast<size_t>(ob(j)) * it.nb[m] + it.r) * 512 +
                                                       lane * 8);
        }
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (((it.who >> (16 * t + n)) & 1ull) && it.r < it.nb[m])
                    v[m][t] = *reinterpret_cast<const f32x4*>(
                        a.v[m] + static_cast<size_t>(i0 + 16 * t + n) * a.max_rank + 16 * it.r + 4 * q);
            }
    };
    u32x2 b0[MB], b1[MB];
    f32x4 v0[NM][4], v1[NM][4];
    bool more = next(nxt);
    if (more) load(nxt, b0, v0);
    while (more) {
        cur = nxt;
        more = next(nxt);
        if (more) load(nxt, b1, v1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (((cur.who >> (16 * t)) & 0xffffull) == 0ull) continue;
            const bool mine = (cur.who >> (16 * t + n)) & 1ull;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const float f[4] = {v0[m][t].x, v0[m][t].y, v0[m][t].z, v0[m][t].w};
                uint32_t terms[VT][2];
                split<VT, 2>(f, terms);
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    if (mat(j) != m) continue;
                    f32x4 sum = acc[j][t];
#pragma unroll
                    for (int k = VT - 1; k >= 0; --k) sum = mma16(b0[j], u32x2{terms[k][0], terms[k][1]}, sum);
                    acc[j][t] = mine ? sum : acc[j][t];   // (a non-finite B stays with its own tokens)
                }
            }
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) b0[j] = b1[j];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) v0[m][t] = v1[m][t];
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
// At most 16 tokens whose adapters hold at most kFusedBlocks rank blocks
// together (bounded by the call's sizes): one launch.  A workgroup owns 16
// outputs (of NM matrices: 2 = gate and up, whose result is silu(g) u).  Its W
// waves take the columns' tiles in turn, of W and of every A in use (each
// workgroup forms A x again: that costs reads from the caches, and saves a
// launch that every output would wait for), and add their sums in LDS in a
// fixed order; B (A x) follows there.
// ---------------------------------------------------------------------------
constexpr int kFusedBlocks = 4;

template <int XK, int YK, int NM, int W, int U>
__global__ __launch_bounds__(W* kWave) void proj_fused_kernel(ProjArgs a) {
    constexpr int TT = Frag<XK>::kTerms, VT = v_terms_for<YK>(), D = kFusedBlocks;
    constexpr int kTiles = NM * (1 + D);   // of matrix m: its outputs, then D products A x
    __shared__ f32x4 part[W][kTiles][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int B_real = real_tokens(a);
    if (B_real <= 0) return;
    const int ob = blockIdx.x, S = a.H / 32;
    const char* w[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m)
        w[m] = static_cast<const char*>(a.w[m]) + static_cast<size_t>(ob) * S * 1024 + lane * 16;
    const char* x = x_row<XK>(a, min(n, B_real - 1), q);

    // the rank blocks in use: A's tiles, B's half tile of these outputs, tokens, scale
    const char* ap[NM][D];
    const char* bp[NM][D];
    uint32_t who[NM][D];
    float scale[NM][D];
    int used[NM];
    const int id = adapter_of(a, n, B_real);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        uint32_t rem = a.table[m] != nullptr ? static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu : 0u, mask = 0u;
        int r = 0, nb = 0;
        moe_lora_handle h;
        used[m] = 0;
#pragma unroll
        for (int d = 0; d < D; ++d) {
            while (r >= nb && rem != 0u) {
                const int ad = __builtin_amdgcn_readlane(id, __ffs(rem) - 1);
                mask = static_cast<uint32_t>(__ballot(id == ad)) & 0xffffu;
                rem &= ~mask;
                h = a.table[m][ad];
                nb = rank_blocks(h, a.max_rank);
                r = 0;
            }
            ap[m][d] = bp[m][d] = nullptr;
            if (r < nb) {
                ap[m][d] = static_cast<const char*>(h.a) + static_cast<size_t>(r) * S * 1024 + lane * 16;
                bp[m][d] = static_cast<const char*>(h.b) + (static_cast<size_t>(ob) * nb + r) * 512 + lane * 8;
                who[m][d] = mask;
                scale[m][d] = h.scale;
                used[m] = d + 1;
                ++r;
            }
        }
    }

    f32x4 acc[NM][1 + D];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int d = 0; d <= D; ++d) acc[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll U
    for (int s = wave; s < S; s += W) {
        const size_t at = static_cast<size_t>(s) * 1024;
        Frag<XK> f;
        f.load(x + static_cast<size_t>(s) * Frag<XK>::kTileBytes, a.x_plane);
        u32x4 t[NM][1 + D], xt[TT];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            t[m][0] = *reinterpret_cast<const u32x4*>(w[m] + at);
#pragma unroll
            for (int d = 0; d < D; ++d) {
                t[m][1 + d] = u32x4{0u, 0u, 0u, 0u};
                if (d < used[m]) t[m][1 + d] = *reinterpret_cast<const u32x4*>(ap[m][d] + at);
            }
        }
        f.terms(xt);
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int d = 0; d <= D; ++d)
#pragma unroll
                for (int k = TT - 1; k >= 0; --k) acc[m][d] = mma32(t[m][d], xt[k], acc[m][d]);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int d = 0; d <= D; ++d)
            if (d <= used[m]) part[wave][m * (1 + D) + d][lane] = acc[m][d];
    __syncthreads();
    for (int p = wave; p < kTiles; p += W) {   // each sum is one wave's, written where only that wave reads
        if (p % (1 + D) > used[NM == 1 ? 0 : p / (1 + D)]) continue;
        f32x4 v = part[0][p][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) v += part[i][p][lane];
        part[0][p][lane] = v;
    }
    __syncthreads();
    if (wave != 0) return;
    f32x4 out[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        out[m] = part[0][m * (1 + D)][lane];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (d >= used[m]) continue;
            f32x4 v = part[0][m * (1 + D) + 1 + d][lane] * scale[m][d];
            const bool mine = (who[m][d] >> n) & 1u;
            const float f[4] = {mine ? v.x : 0.0f, mine ? v.y : 0.0f, mine ? v.z : 0.0f, mine ? v.w : 0.0f};
            uint32_t vt[VT][2];
            split<VT, 2>(f, vt);
            const u32x2 b = *reinterpret_cast<const u32x2*>(bp[m][d]);
            f32x4 sum = out[m];
#pragma unroll
            for (int k = VT - 1; k >= 0; --k) sum = mma16(b, u32x2{vt[k][0], vt[k][1]}, sum);
            out[m] = mine ? sum : out[m];   // (a non-finite B stays with its own tokens)
        }
    }
    if constexpr (NM == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[0][j] = silu(out[0][j]) * out[1][j];
    }
    if (n < B_real) store4<YK>(a, n, 16 * ob + 4 * q, out[0]);
}

// ---------------------------------------------------------------------------
// A decode batch: the columns are split over workgroups too, so that there
// are enough of them, and the adapters' first products run beside the large
// one in the same launch.
//   split launch   workgroups of W waves: first those that form v (shrink),
//                  then those of the product.  One of these owns RB row blocks
//                  (of NM matrices), NT tiles of 16 tokens and one part of the
//                  columns; its waves take pairs of tiles in turn and keep
//                  MB x NT blocks in registers, so a weight tile is read by
//                  one wave only and nothing is staged.  The waves' sums are
//                  added in LDS and stored as 16 x 16 blocks of fp32.  Some
//                  workgroups list, for each tile of 16 tokens, the rank
//                  blocks of B its adapters bring, so that the finish launch
//                  reads the list in place of forming it once per row block.
//   finish launch  a workgroup per few row blocks and token tile: adds the
//                  parts and B v (its waves share both), then the epilogue.
// ---------------------------------------------------------------------------
constexpr int kSplitWaves = 8;
constexpr int kFinishWaves = 8;

// A rank block of one adapter among the tokens of a tile.
struct RankItem {
    const char* b;   // its half tile of row block 0; row block ob lies ob * nb * 512 further
    uint32_t who;    // the adapter's tokens in the tile
    uint16_t nb, r;
};
// An adapter's rank block r is wave (adapter + r) mod kFinishWaves' item, so
// that which wave adds a token's part does not depend on the other tokens: at
// most two of an adapter's 16 rank blocks, for 16 adapters.
constexpr int kMaxItems = 16 * (kMaxLoraRank / 16 / kFinishWaves);

struct SplitArgs {
    f32x4* part;         // [parts][NM][token tiles][row blocks][64]
    RankItem* items;     // [NM][token tiles][kFinishWaves][kMaxItems]
    int* n_items;        // [NM][token tiles][kFinishWaves]
    int parts, steps;    // column tiles per part
    int row_groups, tok_groups;
    int shrink_wgs, places, shrink_parts, by_token;
    int list_wgs;        // one per matrix and token tile, 0: no adapters
};

// The calling wave's list for matrix m and token tile tt.
__device__ __forceinline__ void list_items(const ProjArgs& a, const SplitArgs& g, int m, int tt, int tt_all, int wave,
                                           int B_real) {
    const int lane = threadIdx.x & (kWave - 1);
    const int id = adapter_of(a, 16 * tt + (lane & 15), B_real);
    const size_t at = (static_cast<size_t>(m) * tt_all + tt) * kFinishWaves + wave;
    int nb = 0, count = 0;
    uint64_t base = 0;
    if (a.table[m] != nullptr && id >= 0) {   // every lane reads its own token's handle, all in one round trip
        const moe_lora_handle* h = a.table[m] + id;
        nb = rank_blocks(*h, a.max_rank);
        base = reinterpret_cast<uint64_t>(h->b);
    }
    uint32_t rem = static_cast<uint32_t>(__ballot(nb > 0)) & 0xffffu;
    while (rem != 0u) {
        const int from = __ffs(rem) - 1;
        const int ad = __builtin_amdgcn_readlane(id, from);
        const uint32_t who = static_cast<uint32_t>(__ballot(id == ad)) & 0xffffu;
        rem &= ~who;
        const int n = __builtin_amdgcn_readlane(nb, from);
        const uint64_t b =
            (static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(base >> 32), from)))
             << 32) |
            static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(base), from));
        for (int r = (wave - ad) & (kFinishWaves - 1); r < n; r += kFinishWaves) {
            if (lane == 0)
                g.items[at * kMaxItems + count] = RankItem{reinterpret_cast<const char*>(b) + r * 512, who,
                                                           static_cast<uint16_t>(n), static_cast<uint16_t>(r)};
            ++count;
        }
    }
    if (lane == 0) g.n_items[at] = count;
}

template <int XK, int NM, int NT, int RB>
__global__ __launch_bounds__(kSplitWaves* kWave) void proj_split_kernel(ProjArgs a, SplitArgs g) {
    constexpr int W = kSplitWaves, TT = Frag<XK>::kTerms, MB = NM * RB, T = MB * NT;
    constexpr int SNT = NT == 1 ? 1 : 2;
    union Lds {
        f32x4 part[W / 2][T][kWave];
        char lines[W][NT * 2048];
        ShrinkLds<SNT, 1, W> shrink;
    };
    __shared__ Lds l;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int B_real = real_tokens(a);
    if (static_cast<int>(blockIdx.x) < g.shrink_wgs) {
        const int pieces = a.max_rank / 16;
        const int at = blockIdx.x % g.places, rest = blockIdx.x / g.places;
        const int first = rest % g.shrink_parts, piece = rest / g.shrink_parts;
        const int rb = piece % pieces, t_id = piece / pieces;
        if (a.table[t_id] == nullptr || B_real <= 0) return;
        const int ad = shrink_adapter(a, at, g.by_token, 0, B_real);
        if (ad >= 0) shrink_block<XK, SNT, 1, W>(a, l.shrink, t_id, ad, rb, 0, B_real, first, g.shrink_parts);
        return;
    }
    if (static_cast<int>(blockIdx.x) < g.shrink_wgs + g.list_wgs) {
        const int at = blockIdx.x - g.shrink_wgs, tt_all = (a.B + 15) / 16;
        if (16 * (at % tt_all) < B_real) list_items(a, g, at / tt_all, at % tt_all, tt_all, wave, B_real);
        return;
    }
    const int id = blockIdx.x - g.shrink_wgs - g.list_wgs;
    const int rg = id % g.row_groups, tg = id / g.row_groups % g.tok_groups, sp = id / g.row_groups / g.tok_groups;
    const int i0 = tg * 16 * NT;
    if (i0 >= B_real) return;
    const int ob0 = rg * RB, blocks = a.O / 16, S = a.H / 32;
    const int s0 = sp * g.steps, s1 = min(s0 + g.steps, S);

    const char* wp[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j)
        wp[j] = static_cast<const char*>(a.w[j / RB]) +
                static_cast<size_t>(min(ob0 + j % RB, blocks - 1)) * S * 1024 + lane * 16;
    const char* xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = x_row<XK>(a, min(i0 + 16 * t + n, B_real - 1), q);
    f32x4 acc[T];   // block j NT + t
#pragma unroll
    for (int p = 0; p < T; ++p) acc[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto tile = [&](int s) {
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
                for (int j = 0; j < MB; ++j) acc[j * NT + t] = mma32(w[j], x[k], acc[j * NT + t]);
        }
    };
    if (s1 - s0 >= 2 * W || XK == kActF32) {
        const int pairs = (s1 - s0) / 2;
        constexpr int kU = T * TT > 8 ? 1 : 2;
        if constexpr (XK == kActF32) {
#pragma unroll kU
            for (int p = wave; p < pairs; p += W) {
                tile(s0 + 2 * p);
                tile(s0 + 2 * p + 1);
            }
        } else {
            uint32_t rows[NT][2];   // from the group's first token
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    rows[t][k] = static_cast<uint32_t>(min(16 * t + 8 * k + (lane >> 3), B_real - 1 - i0)) * (a.H * 2) +
                                 (lane & 7) * 16;
            ProjArgs c = a;
            c.x = static_cast<const char*>(a.x) + static_cast<size_t>(i0) * a.H * 2 + static_cast<size_t>(s0) * 64;
            for (int p = wave; p < pairs; p += W * kU) {
                u32x4 w[kU][2][MB];
                Lines<XK, NT> x[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int s = p + u * W;
                    if (s >= pairs) continue;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < MB; ++j)
                            w[u][k][j] =
                                *reinterpret_cast<const u32x4*>(wp[j] + static_cast<size_t>(s0 + 2 * s + k) * 1024);
                    x[u].load(c, rows, s);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    if (p + u * W >= pairs) continue;
#pragma unroll
                    for (int k = Lines<XK, NT>::kParts - 1; k >= 0; --k) {
                        u32x4 f[2][NT];
                        x[u].turn(l.lines[wave], k, f);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int j = 0; j < MB; ++j)
#pragma unroll
                                for (int g = 0; g < 2; ++g)
                                    acc[j * NT + t] = mma32(w[u][g][j], f[g][t], acc[j * NT + t]);
                    }
                }
            }
        }
        if (((s1 - s0) & 1) && wave == W - 1) tile(s1 - 1);
        __syncthreads();   // the lines' room becomes the sums'
    } else {                  // few: a tile for every wave first
        for (int s = s0 + wave; s < s1; s += W) tile(s);
    }
    fold_waves<W>(l.part, acc, wave, lane);
    const int tt_all = (a.B + 15) / 16;
    for (int p = wave; p < T; p += W) {
        const int j = p / NT, t = p % NT, ob = ob0 + j % RB, tt = tg * NT + t;
        if (ob >= blocks || tt >= tt_all) continue;
        f32x4 v = l.part[0][p][lane];
#pragma unroll
        for (int w = 1; w < W / 2; ++w) v += l.part[w][p][lane];
        g.part[(((static_cast<size_t>(sp) * NM + j / RB) * tt_all + tt) * blocks + ob) * kWave + lane] = v;
    }
}

// A workgroup: RBF row blocks (of NM matrices) and one tile of 16 tokens.
template <int YK, int NM, int RBF>
__global__ __launch_bounds__(kFinishWaves* kWave) void proj_finish_kernel(ProjArgs a, SplitArgs g) {
    constexpr int W = kFinishWaves, VT = v_terms_for<YK>(), T = NM * RBF;
    constexpr int D = 4;   // rank blocks in flight per matrix
    __shared__ f32x4 part[W / 2][T][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int n = lane & 15, q = lane >> 4;
    const int tt = blockIdx.y, blocks = a.O / 16, tt_all = gridDim.y, ob0 = blockIdx.x * RBF;
    const int B_real = real_tokens(a);
    if (16 * tt >= B_real) return;
    const int i = 16 * tt + n;
    // The list, then the wave's first part: both on their way while the adapters' operands are fetched.
    u32x4 items[NM];   // lane l holds the wave's item l: one load for the whole list
    int count[NM], most = 0;
#pragma unroll
    for (int m = 0; m < NM; ++m) count[m] = 0;
    if (g.list_wgs > 0) {
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const size_t at = (static_cast<size_t>(m) * tt_all + tt) * W + __builtin_amdgcn_readfirstlane(wave);
            items[m] = *reinterpret_cast<const u32x4*>(g.items + at * kMaxItems + min(lane, kMaxItems - 1));
            count[m] = g.n_items[at];
        }
    }
    auto part_at = [&](int sp, int p) {
        return g.part[(((static_cast<size_t>(sp) * NM + p / RBF) * tt_all + tt) * blocks +
                       min(ob0 + p % RBF, blocks - 1)) * kWave + lane];
    };
    f32x4 acc[T], first[T];   // block m RBF + j
#pragma unroll
    for (int p = 0; p < T; ++p) {
        acc[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        first[p] = wave < g.parts ? part_at(wave, p) : acc[p];
    }
    if (g.list_wgs > 0) {
        const size_t row = static_cast<size_t>(min(i, B_real - 1)) * a.max_rank;
#pragma unroll
        for (int m = 0; m < NM; ++m) most = max(most, count[m]);
        for (int d0 = 0; d0 < most; d0 += D) {   // D items of each matrix, whose loads are in flight together
            u32x2 b[NM][D][RBF];
            f32x4 v[NM][D];
            uint32_t who[NM][D];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    who[m][d] = 0u;
                    if (d0 + d >= count[m]) continue;
                    RankItem it;
                    const uint32_t words[4] = {lane_u32(items[m].x, d0 + d), lane_u32(items[m].y, d0 + d),
                                               lane_u32(items[m].z, d0 + d), lane_u32(items[m].w, d0 + d)};
                    static_assert(sizeof(it) == sizeof(words), "an item is 16 bytes");
                    __builtin_memcpy(&it, words, sizeof(it));
                    who[m][d] = it.who;
#pragma unroll
                    for (int j = 0; j < RBF; ++j)
                        b[m][d][j] = *reinterpret_cast<const u32x2*>(
                            it.b + static_cast<size_t>(min(ob0 + j, blocks - 1)) * it.nb * 512 + lane * 8);
                    v[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    if ((it.who >> n) & 1u)
                        v[m][d] = *reinterpret_cast<const f32x4*>(a.v[m] + row + 16 * it.r + 4 * q);
                }
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (who[m][d] == 0u) continue;
                    const bool mine = (who[m][d] >> n) & 1u;
                    const float f[4] = {v[m][d].x, v[m][d].y, v[m][d].z, v[m][d].w};
                    uint32_t t[VT][2];
                    split<VT, 2>(f, t);
#pragma unroll
                    for (int j = 0; j < RBF; ++j) {
                        f32x4 sum = acc[m * RBF + j];
#pragma unroll
                        for (int k = VT - 1; k >= 0; --k) sum = mma16(b[m][d][j], u32x2{t[k][0], t[k][1]}, sum);
                        // (a non-finite B stays with its own tokens)
                        acc[m * RBF + j] = mine ? sum : acc[m * RBF + j];
                    }
                }
        }
    }
#pragma unroll
    for (int p = 0; p < T; ++p) acc[p] += first[p];
    for (int sp = wave + W; sp < g.parts; sp += W)
#pragma unroll
        for (int p = 0; p < T; ++p) acc[p] += part_at(sp, p);
    fold_waves<W>(part, acc, wave, lane);
    const int ob = ob0 + wave;
    if (wave >= RBF || ob >= blocks || i >= B_real) return;
    f32x4 out[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        out[m] = part[0][m * RBF + wave][lane];
#pragma unroll
        for (int w = 1; w < W / 2; ++w) out[m] += part[w][m * RBF + wave][lane];
    }
    if constexpr (NM == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[0][j] = silu(out[0][j]) * out[1][j];
    }
    store4<YK>(a, i, 16 * ob + 4 * q, out[0]);
}

// ---------------------------------------------------------------------------
// Tiled projection, for many tokens: a workgroup of WR x WC waves owns
// 16 WR MB rows of W (for NM = 2 half of them gate rows and half the up rows of
// the same outputs) and 16 WC NB tokens; a wave owns MB x NB blocks of 16 x 16
// in accumulators.  Operands go to LDS straight from memory (buffer loads to
// LDS): packed weight tiles as they lie, a ring of kWRing steps of 32 columns;
// rows of x as whole 128-byte lines, a ring of kXRing pairs of steps.  (Loading
// x in operand order, 16 bytes from each of 16 rows, touches eight times the
// lines and cost 16 of 127 us at 4096 tokens of 4096 x 4096.)  In LDS the 16-byte
// chunk c of row r lies at place c ^ (r / 2 mod 8) of the row, so that the 16
// rows an operand read takes a chunk from lie in different banks.
//   Step s: wait until this wave's copies up to those of step s - 2 have
//   landed, with them the operands of step s + 1; barrier; start the copies of
//   weight step s + 3 and of half a pair of x, into places whose operands every
//   wave has used by then; read the operands of step s + 1 while the products
//   of step s run: x into a second set of registers, each row of W into the
//   registers its last product has just left.  Copies and reads go between the
//   products; the scheduling barriers keep them there (left to itself the
//   compiler gathers the reads and waits for each).
// Copies past the end take the last step again, so that the waits count alike;
// nothing uses those.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void* lptr;

__device__ __forceinline__ const char* uniform(const char* p) {   // wave-uniform pointer into scalar registers
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const char*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// 16 bytes per lane from base + lane_offset + offset (base and offset uniform)
// to 1 KB at `to` in LDS.  A buffer load: the compiler waits for LDS reads all
// together where a global load to LDS is in flight, and one by one here.
__device__ __forceinline__ void copy_tile(const char* base, int lane_offset, int offset, char* to) {
#ifdef __HIP_DEVICE_COMPILE__   // (the resource type does not exist in the host pass)
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0x7fffffff, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr)to, 16, lane_offset, offset, 0, 0);
#endif
}

constexpr int kWRing = 4, kXRing = 3;

// At most N vector-memory operations of this wave still in flight; then the
// workgroup's barrier.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int XK, int YK, int NM, int WR, int WC, int MB, int NB>
__global__ __launch_bounds__(WR* WC* kWave, 2) void proj_tile_kernel(ProjArgs a, int row_tiles, int tok_tiles) {
    constexpr int NW = WR * WC;
    constexpr int RT = WR * MB, CT = WC * NB;         // row and token blocks of the workgroup
    constexpr int kPerW = RT / NW, kPerX = CT / NW;   // KB a wave copies per step (of x: kPerX in each step of a pair)
    constexpr int kPer = kPerW + kPerX;
    static_assert(RT % NW == 0 && CT % NW == 0 && MB % NM == 0 && NB % 4 == 0 && MB % kPer == 0, "tile split");
    constexpr int P = XK == kActPlanes ? 3 : 1;
    constexpr int kXPair = 2 * CT * 1024;
    __shared__ __align__(1024) char lds[kWRing * RT * 1024 + kXRing * kXPair];
    char* const lds_x = lds + kWRing * RT * 1024;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, q = lane >> 4;
    const int wr = wave / WC, wc = wave % WC;
    const int B_real = real_tokens(a);
    // Workgroup id mod 8 is the XCD: each XCD gets a contiguous run of tiles,
    // in bands of four row tiles, so that its L2 holds what they share.
    const int all = row_tiles * tok_tiles, xcd = blockIdx.x & 7;
    const int at = xcd * (all >> 3) + min(xcd, all & 7) + (static_cast<int>(blockIdx.x) >> 3);
    const int band = at / (4 * tok_tiles), in = at - band * 4 * tok_tiles, wide = min(4, row_tiles - 4 * band);
    const int tile_r = 4 * band + in % wide, tile_c = in / wide;
    const int i0 = tile_c * 16 * CT;
    if (i0 >= B_real) return;
    const int blocks = a.O / 16, S = a.H / 32;
    const int ob0 = tile_r * (RT / NM);
    // output row block and matrix of row tile j of the workgroup
    constexpr int kHalf = MB / NM;
    auto mat_of = [](int j) { return NM == 1 ? 0 : (j % MB) / kHalf; };
    auto ob_of = [&](int j) { return min(ob0 + (NM == 1 ? j : (j / MB) * kHalf + j % kHalf), blocks - 1); };

    const char* w_base[kPerW];
#pragma unroll
    for (int u = 0; u < kPerW; ++u) {
        const int j = wave * kPerW + u;
        w_base[u] = uniform(static_cast<const char*>(mat_of(j) ? a.w[1] : a.w[0]) +
                            static_cast<size_t>(ob_of(j)) * S * 1024);
    }
    // x: copy g of a pair takes 8 rows of 128 bytes, lane l chunk (l % 8 ^ swizzle) of row 8 g + l / 8
    const char* x_base = uniform(static_cast<const char*>(a.x) + static_cast<size_t>(i0) * a.H * 2);
    int x_at[2][kPerX], x_chunk[2][kPerX];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < kPerX; ++u) {
            const int r = 8 * ((2 * wave + h) * kPerX + u) + (lane >> 3);   // row of the workgroup's tokens
            x_chunk[h][u] = (lane & 7) ^ ((r >> 1) & 7);
            x_at[h][u] = (min(i0 + r, B_real - 1) - i0) * a.H * 2 + 16 * x_chunk[h][u];   // (at most 256 rows of 32 KB)
        }
    auto copy_w = [&](int step, int u) {
        copy_tile(w_base[u], lane * 16, min(step, S - 1) * 1024,
                  lds + (step % kWRing) * RT * 1024 + (wave * kPerW + u) * 1024);
    };
    const int last_pair = (S - 1) / 2;
    auto copy_x = [&](int pair, int place, int h, int u) {
        // (the last pair of an odd number of steps is half a line)
        const int back = pair >= last_pair && (S & 1) && x_chunk[h][u] >= 4 ? 64 : 0;
        copy_tile(x_base, x_at[h][u] - back, min(pair, last_pair) * 128,
                  lds_x + place * kXPair + ((2 * wave + h) * kPerX + u) * 1024);
    };

    constexpr int Q = NB / 4;   // runs of 64 tokens
    f32x4 acc[Q][MB][4];
#pragma unroll
    for (int h = 0; h < Q; ++h)
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[h][j][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const char* mine_w = lds + wr * MB * 1024 + lane * 16;
    const char* mine_x[2];   // by the step's place in its pair
#pragma unroll
    for (int h = 0; h < 2; ++h)
        mine_x[h] = lds_x + wc * NB * 2048 + n * 128 + (((4 * h + q) ^ ((n >> 1) & 7)) * 16);

    for (int plane = P - 1; plane >= 0; --plane) {   // the smallest term first
        if (P > 1)
            x_base = uniform(static_cast<const char*>(a.x) + static_cast<size_t>(plane) * a.x_plane +
                             static_cast<size_t>(i0) * a.H * 2);
        int p0 = 0, p1 = 1, p2 = 2;   // places of pairs p, p + 1, p + 2
#pragma unroll
        for (int u = 0; u < 2 * kPerX; ++u) copy_x(0, 0, u / kPerX, u % kPerX);
#pragma unroll
        for (int u = 0; u < 2 * kPerW; ++u) copy_w(u / kPerW, u % kPerW);
#pragma unroll
        for (int u = 0; u < 2 * kPerX; ++u) copy_x(1, 1, u / kPerX, u % kPerX);
#pragma unroll
        for (int u = 0; u < kPerW; ++u) copy_w(2, u);
        wait_and_barrier<2 * kPerX + 2 * kPerW>();   // pair 0 and weight step 0 are there
        u32x4 w[MB], x0[NB], x1[NB];
#pragma unroll
        for (int t = 0; t < NB; ++t) x0[t] = *reinterpret_cast<const u32x4*>(mine_x[0] + t * 2048);
#pragma unroll
        for (int j = 0; j < MB; ++j) w[j] = *reinterpret_cast<const u32x4*>(mine_w + j * 1024);
        // step s, the h-th of its pair: x_next holds the pair that step s + 1 is in
        auto step = [&](int s, int h, int x_next, const u32x4 (&x)[NB], u32x4 (&xn)[NB]) {
            wait_and_barrier<kPer>();
            __builtin_amdgcn_sched_barrier(0);
            const char* from_w = mine_w + ((s + 1) % kWRing) * RT * 1024;
            const char* from_x = mine_x[h ^ 1] + x_next * kXPair;
#pragma unroll
            for (int j = 0; j < MB; ++j) {
#pragma unroll
                for (int t = j * NB / MB; t < (j + 1) * NB / MB; ++t)
                    xn[t] = *reinterpret_cast<const u32x4*>(from_x + t * 2048);
#pragma unroll
                for (int t = 0; t < NB; ++t) acc[t / 4][j][t % 4] = mma32(w[j], x[t], acc[t / 4][j][t % 4]);
                w[j] = *reinterpret_cast<const u32x4*>(from_w + j * 1024);
                if (j % (MB / kPer) == MB / kPer - 1) {
                    const int u = j / (MB / kPer);
                    if (u < kPerW) copy_w(s + 3, u);
                    else copy_x(s / 2 + 2, p2, h, u - kPerW);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        for (int s = 0; s + 1 < S; s += 2) {
            step(s, 0, p0, x0, x1);
            step(s + 1, 1, p1, x1, x0);
            const int p = p0;
            p0 = p1;
            p1 = p2;
            p2 = p;
        }
        if (S & 1)
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int t = 0; t < NB; ++t) acc[t / 4][j][t % 4] = mma32(w[j], x0[t], acc[t / 4][j][t % 4]);
        // No copy may land in the next plane's ring, or after the workgroup's end, and none of the next plane's
        // before a wave has its last operands.
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
#pragma unroll
    for (int h = 0; h < Q; ++h) {
        const int i1 = i0 + 16 * NB * wc + 64 * h;
        expand<v_terms_for<YK>(), NM>(a, i1, B_real, acc[h], [&](int j) { return ob_of(wr * MB + j); },
                                  [&](int j) { return mat_of(j); });
#pragma unroll
        for (int j = 0; j < kHalf; ++j) {
            const int ob = ob0 + wr * kHalf + j;
            if (ob >= blocks) continue;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int i = i1 + 16 * t + n;
                f32x4 r = acc[h][j][t];
                if constexpr (NM == 2) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) r[e] = silu(r[e]) * acc[h][j + kHalf][t][e];
                }
                if (i < B_real) store4<YK>(a, i, 16 * ob + 4 * q, r);
            }
        }
    }
}

// fp32 rows (the real tokens') cut into their three bf16 terms, as planes.
__global__ __launch_bounds__(256) void planes_kernel(ProjArgs a, u32x2* __restrict__ out, size_t plane) {
    const f32x4* x = static_cast<const f32x4*>(a.x);
    const long chunks = static_cast<long>(real_tokens(a)) * a.H / 4;
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

// ---------------------------------------------------------------------------
// Which kernels a projection takes, from its sizes alone.
// ---------------------------------------------------------------------------
constexpr int kRowTokens = 16;       // up to this many: fp32 rows are cut in registers
enum Path { kFused, kSplit, kTiled };
struct Plan {
    Path path;
    int nt, rb;          // split: token tiles and row blocks of a workgroup
    SplitArgs split;
    size_t part_bytes, item_bytes, count_bytes;
};

// rank_blocks: what the batch's adapters may hold together (0: no adapters);
// terms: bf16 terms an activation enters with.
Plan plan_proj(int B, int H, int O, int mats, int rank_blocks, int terms) {
    Plan p{};
    if (B <= 16 && rank_blocks <= kFusedBlocks) {
        p.path = kFused;
        return p;
    }
    p.path = kSplit;
    p.nt = B <= 16 ? 1 : (B <= 32 ? 2 : 4);
    p.rb = (p.nt == 4 ? 4 : 2) / mats;   // (as the instances in launch_proj)
    const int blocks = O / 16, S = H / 32;
    SplitArgs& g = p.split;
    g.row_groups = (blocks + p.rb - 1) / p.rb;
    g.tok_groups = (B + 16 * p.nt - 1) / (16 * p.nt);
    // a workgroup per compute unit (two: 14.4 against 11.6 us for 64 tokens of 4096 x 4096, more partial
    // blocks to write and add), but at least a pair of tiles per wave
    const long groups = static_cast<long>(g.row_groups) * g.tok_groups;
    const int want = static_cast<int>(std::max(1L, 256 / groups));
    const int most = std::max(1, S / (2 * kSplitWaves));
    g.parts = std::min(want, most);
    g.steps = (S + g.parts - 1) / g.parts;
    g.steps += g.steps & 1;
    g.parts = (S + g.steps - 1) / g.steps;
    if (B > 64) {
        // Split or tiled, by what 96 sizes of H 512-4096, O 256-4096 and B 65-4096 measured, in ns (within 20 %).
        // Split: 3 us and, for each workgroup on a compute unit, 5.5 us and 127 ns per step of 32 columns
        // (4096 x 1024, B = 512: 19 us against 35 tiled).  Tiled: 3.3 us and 250 ns per step, which two workgroups
        // on a unit share well (B = 4096 of the same: 98 split, 39 tiled).  Adapters cost the tiled path a launch
        // before and the rank blocks behind its products.
        const long rounds = (groups * g.parts + 255) / 256;
        const long tiles = (static_cast<long>(O) * mats + 127) / 128 * ((B + 127) / 128);
        const long split_ns = 3000 + rounds * (5500 + 127L * g.steps * (terms > 1 ? 2 : 1));
        const long tile_ns = 3300 + 250L * S * terms * std::max(100L, 35 + 65 * tiles / 256) / 100 +
                             (rank_blocks > 0 ? 6000 : 0);
        if (B > kChunk || tile_ns < split_ns) {   // (the split launch forms v over one chunk of tokens)
            p.path = kTiled;
            return p;
        }
    }
    const size_t lists = static_cast<size_t>(mats) * ((B + 15) / 16) * kFinishWaves;
    p.part_bytes = static_cast<size_t>(g.parts) * mats * ((B + 15) / 16) * blocks * 1024;
    p.item_bytes = lists * kMaxItems * sizeof(RankItem);
    p.count_bytes = lists * sizeof(int);
    return p;
}
int rank_blocks_bound(int B, int n_adapters, int max_rank) { return std::min(B, n_adapters) * (max_rank / 16); }

template <int XK, int YK, int NM, int WR, int WC, int MB, int NB>
hipError_t launch_tile(const ProjArgs& a, hipStream_t s) {
    constexpr int kRows = 16 * WR * MB / NM, kTok = 16 * WC * NB;
    const int rt = (a.O + kRows - 1) / kRows, ct = (a.B + kTok - 1) / kTok;
    proj_tile_kernel<XK, YK, NM, WR, WC, MB, NB><<<static_cast<unsigned>(rt) * ct, WR * WC * kWave, 0, s>>>(a, rt, ct);
    return hipGetLastError();
}

template <int XK, int NM, int NT, int RB>
void launch_split(const ProjArgs& a, const SplitArgs& g, hipStream_t s) {
    const long wgs = static_cast<long>(g.row_groups) * g.tok_groups * g.parts + g.shrink_wgs + g.list_wgs;
    proj_split_kernel<XK, NM, NT, RB><<<static_cast<unsigned>(wgs), kSplitWaves * kWave, 0, s>>>(a, g);
}

template <int XK>
void launch_shrink(const ProjArgs& a, int tables, hipStream_t s) {
    constexpr int NT = 2, RBN = 2, W = 8;
    const int chunk = std::min(a.B, kChunk), chunks = (a.B + kChunk - 1) / kChunk;
    const int by_token = a.n_adapters > chunk, places = by_token ? chunk : a.n_adapters;
    // workgroups per place: with tokens spread evenly each has a part or two; more tokens take turns
    const int parts = std::max(1, std::min((chunk + 16 * NT - 1) / (16 * NT), 128 / places));
    const int pieces = (a.max_rank / 16 + RBN - 1) / RBN;
    shrink_kernel<XK, NT, RBN, W>
        <<<dim3(places, parts * chunks, pieces * tables), W * kWave, 0, s>>>(a, parts, by_token);
}

// One projection (NM = 1) or the gate/up pair (NM = 2).
template <int XK, int YK, int NM>
hipError_t launch_proj(const ProjArgs& a, void* part, hipStream_t s) {
    const bool lora = a.adapter != nullptr && (a.table[0] != nullptr || (NM == 2 && a.table[1] != nullptr));
    Plan p = plan_proj(a.B, a.H, a.O, NM, a.adapter != nullptr ? rank_blocks_bound(a.B, a.n_adapters, a.max_rank) : 0,
                       XK == kActBf16 ? 1 : 3);
    if (p.path == kFused) {
        // 16 waves where each has four steps and more (H = 2048, one token: 5.7 against 6.3 us; H = 768: 4.7 against
        // 4.1)
        if (a.H >= 2048) proj_fused_kernel<XK, YK, NM, 16, 4><<<a.O / 16, 16 * kWave, 0, s>>>(a);
        else proj_fused_kernel<XK, YK, NM, 8, 4><<<a.O / 16, 8 * kWave, 0, s>>>(a);
        return hipGetLastError();
    }
    if (p.path == kSplit) {
        SplitArgs& g = p.split;
        char* lists = static_cast<char*>(part) + p.part_bytes;
        g.part = static_cast<f32x4*>(part);
        g.items = reinterpret_cast<RankItem*>(lists);
        g.n_items = reinterpret_cast<int*>(lists + p.item_bytes);
        if (lora) {
            g.by_token = a.n_adapters > a.B;
            g.places = g.by_token ? a.B : a.n_adapters;
            // workgroups per place and rank block: with tokens spread evenly one part each; more tokens take turns
            g.shrink_parts = std::max(1, std::min((a.B + 31) / 32, 32 / g.places));
            g.shrink_wgs = g.places * g.shrink_parts * (a.max_rank / 16) * NM;
            g.list_wgs = NM * ((a.B + 15) / 16);
        }
        if (p.nt == 1) launch_split<XK, NM, 1, 2 / NM>(a, g, s);
        else if constexpr (XK != kActF32) {
            if (p.nt == 2) launch_split<XK, NM, 2, 2 / NM>(a, g, s);
            else launch_split<XK, NM, 4, 4 / NM>(a, g, s);
        }
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int blocks = a.O / 16, tts = (a.B + 15) / 16;
        if (blocks * tts >= 512)
            proj_finish_kernel<YK, NM, 4><<<dim3((blocks + 3) / 4, tts), kFinishWaves * kWave, 0, s>>>(a, g);
        else
            proj_finish_kernel<YK, NM, 1><<<dim3(blocks, tts), kFinishWaves * kWave, 0, s>>>(a, g);
        return hipGetLastError();
    }
    if constexpr (XK != kActF32) {
        if (lora) {
            launch_shrink<XK>(a, NM, s);
            hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        // 128 x 128 tiles, two workgroups on a compute unit, up to three rounds of units (512 tiles of H = 4096: 65 us
        // against 83); 256 x 256 beyond (1024: 109 against 130).  The gate/up pair turns earlier (576: 111 against
        // 100).
        const long tiles = (static_cast<long>(a.O) * NM + 127) / 128 * ((a.B + 127) / 128);
        return tiles < (NM == 2 ? 576 : 768) ? launch_tile<XK, YK, NM, 2, 2, 4, 4>(a, s)
                                             : launch_tile<XK, YK, NM, 2, 4, 8, 4>(a, s);
    }
    return hipErrorInvalidValue;
}

template <int NM>
hipError_t run_proj(const ProjArgs& a, void* part, hipStream_t s) {
#define MOE_PROJ(X_, Y_) \
    if (a.x_kind == X_ && a.y_kind == Y_) return launch_proj<X_, Y_, NM>(a, part, s)
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
// How the shared expert's h is kept: as the three terms of its fp32 value for
// an fp32 y, and for a bf16 y of up to 32 tokens, which are bound by latency;
// beyond, rounded to bf16 once, as y is (101 tokens of H = 1344, I = 1280: 25 us
// against 32 with three terms).
bool h_is_cut(int B, bool y_f32) { return y_f32 || B <= 32; }

// Partial blocks and item lists of a projection: the most any number of
// adapters asks for.
size_t part_bytes(int B, int H, int O, int mats, int max_rank, int x_dtype) {
    const Plan p = plan_proj(B, H, O, mats, max_rank > 0 ? kFusedBlocks + 1 : 0, x_dtype == MOE_DT_F32 ? 3 : 1);
    return up256(p.part_bytes + p.item_bytes + p.count_bytes);
}

// Cut an fp32 x into planes at `ws` where the call's kernels read planes.
hipError_t cut_x(ProjArgs& a, void* ws, hipStream_t s) {
    if (a.x_kind != kActF32 || a.B <= kRowTokens) return hipSuccess;
    const size_t plane = up256(static_cast<size_t>(a.B) * a.H * 2);
    const long chunks = static_cast<long>(a.B) * a.H / 4;
    planes_kernel<<<static_cast<unsigned>(std::min<long>((chunks + 255) / 256, 4096)), 256, 0, s>>>(
        a, static_cast<u32x2*>(ws), plane);
    a.x = ws;
    a.x_kind = kActPlanes;
    a.x_plane = plane;
    return hipGetLastError();
}

}  // namespace

// v, the planes of x, partial blocks.
size_t lora_workspace_bytes(int B, int H, int O, int max_rank, int x_dtype) {
    return v_bytes(B, max_rank) + x_planes_bytes(B, H, x_dtype) + part_bytes(B, H, O, 1, max_rank, x_dtype);
}

// v of gate, up and down, the planes of x, h (bf16 or three planes), partial
// blocks of the larger projection.
size_t shared_ffn_workspace_bytes(int B, int H, int I, int max_rank, int x_dtype, int y_dtype) {
    const bool cut = h_is_cut(B, y_dtype == MOE_DT_F32);
    return 3 * v_bytes(B, max_rank) + x_planes_bytes(B, H, x_dtype) +
           (cut ? 3 : 1) * up256(static_cast<size_t>(B) * I * 2) +
           std::max(part_bytes(B, H, I, 2, max_rank, x_dtype),
                    part_bytes(B, I, H, 1, max_rank, cut ? MOE_DT_F32 : MOE_DT_BF16));
}

hipError_t launch_lora_linear(ProjArgs a, void* ws, hipStream_t s) {
    char* p = static_cast<char*>(ws);
    a.v[0] = static_cast<float*>(ws);
    char* planes = p + v_bytes(a.B, a.max_rank);
    char* part = planes + x_planes_bytes(a.B, a.H, a.x_kind == kActF32 ? MOE_DT_F32 : MOE_DT_BF16);
    hipError_t e = cut_x(a, planes, s);
    return e != hipSuccess ? e : run_proj<1>(a, part, s);
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
    a.y_kind = h_is_cut(a.B, a.y_kind == kActF32) ? kActPlanes : kActBf16;
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
    char* part = h + (a.y_kind == kActPlanes ? 3 : 1) * h_plane;
    hipError_t e = cut_x(a, x_planes, s);
    if (e == hipSuccess) e = run_proj<2>(a, part, s);
    return e != hipSuccess ? e : run_proj<1>(d, part, s);
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

// paged_attention.hip -- attention of a chunk of new tokens (one for a draft step, gamma + 1 for
// a verify step, thousands for a prompt) over the paged key/value cache, for gfx950.
//
// Query i of a sequence with n new tokens and L cached ones (the new ones among them) sits at
// position p = L - n + i and sees the keys 0..p:
//     out = sum_j softmax_j(scale * q . k_j) v_j
// A row that sees no key gives 0.  Query heads g * kv_head .. share a key/value head: the
// rows of a key/value head are its n * G (query, head) pairs, query-major, so that all of them
// use each key and value that is read.
//
// The softmax is taken in one pass over the keys with a running maximum and sum, in base 2 with
// scale * log2(e) folded into one multiplication.  Scores, maxima, sums and outputs are
// binary32; the weights are rounded to bfloat16 for the matrix cores (2^-9 relative each, against
// outputs that are rounded to bfloat16 themselves).  8-bit codes are exact in bfloat16: a
// key's scale multiplies its score, a value's scale its weight.
#include "internal.h"

using namespace w4host;
using namespace w4dev;

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 32;        // tokens of one step
constexpr float kLag = 8.0f;      // log2 by which a running maximum may lag
constexpr float kNone = -__builtin_huge_valf();

struct AttnParams {
    const uint16_t *q;
    int64_t q_tok_stride, q_head_stride;
    const void *k, *v;
    const float *ks, *vs;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *q_start, *kv_len;
    uint16_t *out;
    float *part;       // [splits][T * Hq][D] unnormalized outputs
    float *part_ml;    // [splits][T * Hq][2] running maximum and sum
    float scale2;      // scale * log2(e)
    int Hq, Hkv, G, T, width, pages, page_tiles, splits;
    uint64_t page_magic;  // ceil(2^32 / page_tiles)
    int q_vec;
};

// One sequence's chunk: first row of q, new tokens, cached tokens.  Offsets outside [0, T] or out
// of order are cut to what lies inside, so that no access depends on them.
struct Seq {
    int start, n, kv;
};
__device__ __forceinline__ Seq seq_of(const AttnParams &p, int b)
{
    Seq s;
    s.start = min(max(p.q_start[b], 0), p.T);
    s.n = min(max(p.q_start[b + 1], s.start), p.T) - s.start;
    s.kv = max(p.kv_len[b], 0);
    return s;
}

// How a row block's `blocks` steps are shared out: `per` for each split but the last used one.
struct Share {
    int per, used;
};
__device__ __forceinline__ Share share_of(int tokens, int splits, int waves)
{
    const int blocks = (tokens + kBlock - 1) / kBlock;
    Share s;
    s.per = max(1, ((blocks + splits - 1) / splits + waves - 1) / waves * waves);
    s.used = max(1, (blocks + s.per - 1) / s.per);
    return s;
}

// Keys that a row block sees: those up to its last row's position.
__device__ __forceinline__ int tokens_of(const Seq &s, int last_row, int G)
{
    return max(0, s.kv - s.n + last_row / G + 1);
}

__device__ __forceinline__ f32x4 mfma16(const u32x4 &a, const u32x4 &b, const f32x4 &c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Four signed bytes to two bfloat16 pairs, exactly.
__device__ __forceinline__ float sbyte(uint32_t w, int j) { return (float)(int8_t)(w >> (8 * j)); }

// ------------------------------------------------------------------------------------
// Few rows: keys and values from HBM straight to registers.
//
// A workgroup of 4 waves takes up to 16 * RT rows of one key/value head and a range of its tokens;
// each wave walks steps of 32 tokens (two 16-token tiles; a tile lies in one page).
//   S^T = K Q^T:  lane l holds the 16 bytes of token l % 16 that operand A wants, and gets the
//     scores of row l % 16 for tokens 4 (l / 16) + 0..3 of each tile.
//   O^T = V^T P^T: those 8 weights are operand B as they are, if operand A's k slots are the same 8
//     tokens.  So a lane loads V rows of its 8 tokens, columns (l % 16) * D/16 .., and a column's
//     pairs of tokens are put together by one byte permute a pair; no LDS, no cross-lane move.
// Each lane's accumulators belong to its own row (l % 16), so a new maximum rescales them in
// place.  The maximum is allowed to lag by 2^8 behind the scores: then a step needs no reduction
// over lanes, only a vote, and the sum stays per lane until the end.
template <int D, bool I8>
struct KeyRegs {
    u32x4 k[2][D / 32];      // bf16: operand per 32-wide step; 8-bit: [tile][D / 64] used
    f32x4 s[2];              // 8-bit: scales of the lane's score rows
};
template <int D, bool I8>
struct ValueRegs {
    uint32_t v[8][I8 ? D / 64 : D / 32];
    f32x4 s[2];
};

template <int D, bool I8, int RT>
__global__ __launch_bounds__(256, RT <= 2 ? 2 : 1) void attn_rows_kernel(const AttnParams p)
{
    constexpr int kSteps = D / 32;        // k-steps of the scores
    constexpr int kCols = D / 16;         // columns of V a lane holds = output tiles
    constexpr int kRowPad = D + 4;
    __shared__ __align__(16) float s_o[4][16 * kRowPad];
    __shared__ float s_m[4][16 * RT], s_l[4][16 * RT];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, quad = lane >> 4;
    const int split = blockIdx.x % p.splits, rb = blockIdx.x / p.splits, h = blockIdx.y, b = blockIdx.z;
    const Seq sq = seq_of(p, b);
    const int rows = sq.n * p.G, r0 = rb * 16 * RT;
    if (r0 >= rows) return;
    const int last = min(rows, r0 + 16 * RT) - 1;
    const int tokens = tokens_of(sq, last, p.G);
    const Share sh = share_of(tokens, p.splits, 4);
    if (split >= sh.used) return;
    const int blocks = (tokens + kBlock - 1) / kBlock;
    const int blk_end = min(blocks, (split + 1) * sh.per);
    const int first_pos = sq.kv - sq.n + r0 / p.G;   // the least position of the rows

    // queries: row c of each row tile, the columns of operand B's step
    u32x4 qf[RT][kSteps];
    int pos[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        const int r = min(r0 + 16 * rt + c, rows - 1);
        const int i = r / p.G, g = r - i * p.G;
        pos[rt] = sq.kv - sq.n + i;
        const uint16_t *src = p.q + (int64_t)(sq.start + i) * p.q_tok_stride + (int64_t)(h * p.G + g) * p.q_head_stride;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            // 8-bit keys come 16 codes a lane: columns 64 (s/2) + 16 quad + 8 (s%2) ..
            const int d = I8 ? 64 * (s >> 1) + 16 * quad + 8 * (s & 1) : 32 * s + 8 * quad;
            if (p.q_vec) {
                qf[rt][s] = *(const u32x4 *)(src + d);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    qf[rt][s][j] = (uint32_t)src[d + 2 * j] | (uint32_t)src[d + 2 * j + 1] << 16;
            }
        }
    }

    f32x4 acc[RT][kCols];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) acc[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        m[rt] = kNone;
        l[rt] = 0.f;
    }

    // The place of a 16-token tile: row index of its first token in the cache, or -1.
    auto tile_row = [&](int tile) -> int64_t {
        const int page = (int)((uint64_t)(uint32_t)tile * p.page_magic >> 32);
        int id = -1;
        if (page < p.width) id = p.table[(int64_t)b * p.table_stride + page];
        if (id < 0 || id >= p.pages) return -1;
        return ((int64_t)id * p.Hkv + h) * (p.page_tiles * 16) + (tile - page * p.page_tiles) * 16;
    };
    const int last_tile = (tokens - 1) / 16;
    auto rows_of = [&](int blk, int64_t (&row)[2]) {
        row[0] = tile_row(min(2 * blk, last_tile));
        row[1] = tile_row(min(2 * blk + 1, last_tile));
    };
    auto load_k = [&](const int64_t (&row)[2], KeyRegs<D, I8> &kr) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t at = row[t] < 0 ? 0 : row[t];
            if constexpr (I8) {
                const uint8_t *src = (const uint8_t *)p.k + at * D;
#pragma unroll
                for (int s = 0; s < D / 64; ++s) kr.k[t][s] = *(const u32x4 *)(src + c * D + 64 * s + 16 * quad);
                kr.s[t] = *(const f32x4 *)(p.ks + at + 4 * quad);
            } else {
                const uint16_t *src = (const uint16_t *)p.k + at * D;
#pragma unroll
                for (int s = 0; s < kSteps; ++s) kr.k[t][s] = *(const u32x4 *)(src + c * D + 32 * s + 8 * quad);
            }
        }
    };
    auto load_v = [&](const int64_t (&row)[2], ValueRegs<D, I8> &vr) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t at = row[t] < 0 ? 0 : row[t];
            const char *src = (const char *)p.v + at * D * (I8 ? 1 : 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const char *a = src + ((4 * quad + e) * D + c * kCols) * (I8 ? 1 : 2);
                if constexpr (!I8 && D == 128) {
                    const u32x4 x = *(const u32x4 *)a;
#pragma unroll
                    for (int j = 0; j < 4; ++j) vr.v[4 * t + e][j] = x[j];
                } else if constexpr (I8 && D == 64) {
                    vr.v[4 * t + e][0] = *(const uint32_t *)a;
                } else {
                    const u32x2 x = *(const u32x2 *)a;
                    vr.v[4 * t + e][0] = x[0];
                    vr.v[4 * t + e][1] = x[1];
                }
            }
            if constexpr (I8) vr.s[t] = *(const f32x4 *)(p.vs + at + 4 * quad);
        }
    };

    auto step = [&](int blk, const int64_t (&row)[2], const KeyRegs<D, I8> &kr, ValueRegs<D, I8> &vr) {
        const int t0 = blk * kBlock;
        const bool masked = t0 + kBlock - 1 > first_pos;       // some row does not see some token
        const bool bad0 = row[0] < 0, bad1 = row[1] < 0;
        u32x4 pf[RT];
        f32x4 sc[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sc[rt][0] = sc[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                u32x4 a;
                if constexpr (I8) {
                    const uint32_t w0 = kr.k[t][s >> 1][2 * (s & 1)], w1 = kr.k[t][s >> 1][2 * (s & 1) + 1];
                    a = u32x4{pack_bf16(sbyte(w0, 0), sbyte(w0, 1)), pack_bf16(sbyte(w0, 2), sbyte(w0, 3)),
                              pack_bf16(sbyte(w1, 0), sbyte(w1, 1)), pack_bf16(sbyte(w1, 2), sbyte(w1, 3))};
                } else {
                    a = kr.k[t][s];
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sc[rt][t] = mfma16(a, qf[rt][s], sc[rt][t]);
            }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = I8 ? kr.s[e >> 2][e & 3] * p.scale2 : p.scale2;
                x[e] = sc[rt][e >> 2][e & 3] * f;
            }
            if (bad0 || bad1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < 4 ? bad0 : bad1) x[e] = __builtin_nanf("");
            }
            if (masked) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (t0 + 16 * (e >> 2) + 4 * quad + (e & 3) > pos[rt]) x[e] = kNone;
            }
            float mx = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, x[e]);
            if (__any(mx > m[rt] + kLag)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                mx = fmaxf(mx, m[rt]);
                const float f = mx == kNone ? 1.f : exp2_fast(m[rt] - mx);
                m[rt] = mx;
                l[rt] *= f;
#pragma unroll
                for (int j = 0; j < kCols; ++j) acc[rt][j] *= f;
            }
            const float base = m[rt] == kNone ? 0.f : m[rt];
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[e] = exp2_fast(x[e] - base);
                l[rt] += w[e];
            }
            if constexpr (I8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float y = w[e] * vr.s[e >> 2][e & 3];
                    w[e] = masked && x[e] == kNone ? 0.f : y;   // an unseen token's scale may be anything
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) pf[rt][e] = pack_bf16(w[2 * e], w[2 * e + 1]);
        }
        bool wild = false;
        if constexpr (!I8) {
            if (masked || bad0 || bad1) {
                // What lies behind the sequence's end in its last page, and what a bad page number
                // stands for, may be anything: cleared.  A value that some row does not see may
                // be infinite or NaN, which a weight of 0 does not take away: set aside.
                uint32_t odd = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool none = (e < 4 ? bad0 : bad1) || t0 + 16 * (e >> 2) + 4 * quad + (e & 3) >= sq.kv;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        if (none) vr.v[e][j] = 0u;
                        odd |= (vr.v[e][j] & 0x7F80u) == 0x7F80u;
                        odd |= (vr.v[e][j] & 0x7F800000u) == 0x7F800000u;
                    }
                }
                wild = __any(odd);
            }
        }
        if constexpr (!I8) {
            if (wild) {
                // Each kind of such values by itself: which of them a row sees is a product of two
                // 0/1 matrices, and a row that sees one gets it.
                for (int kind = 0; kind < 3; ++kind) {
                    auto is = [&](uint32_t x) -> uint32_t {  // 1.0 in bfloat16 where x is of this kind
                        const bool y = kind == 0 ? (x & 0x7FFFu) > 0x7F80u : x == (kind == 1 ? 0x7F80u : 0xFF80u);
                        return y ? 0x3F80u : 0u;
                    };
                    const float value = kind == 0 ? __builtin_nanf("") : kind == 1 ? -kNone : kNone;
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        u32x4 seen;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = t0 + 16 * (e >> 1) + 4 * quad + 2 * (e & 1);
                            seen[e] = (tok <= pos[rt] ? 0x3F80u : 0u) | (tok + 1 <= pos[rt] ? 0x3F800000u : 0u);
                        }
#pragma unroll
                        for (int j = 0; j < kCols; ++j) {
                            u32x4 a;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                a[e] = is((vr.v[2 * e][j >> 1] >> (16 * (j & 1))) & 0xFFFFu) |
                                       is((vr.v[2 * e + 1][j >> 1] >> (16 * (j & 1))) & 0xFFFFu) << 16;
                            const f32x4 n = mfma16(a, seen, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (n[i] > 0.f) acc[rt][j][i] += value;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) {
                        if ((vr.v[e][j] & 0x7F80u) == 0x7F80u) vr.v[e][j] &= 0xFFFF0000u;
                        if ((vr.v[e][j] & 0x7F800000u) == 0x7F800000u) vr.v[e][j] &= 0xFFFFu;
                    }
            }
        }
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            u32x4 a;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (I8)
                    a[e] = pack_bf16(sbyte(vr.v[2 * e][j >> 2], j & 3), sbyte(vr.v[2 * e + 1][j >> 2], j & 3));
                else
                    a[e] = __builtin_amdgcn_perm(vr.v[2 * e + 1][j >> 1], vr.v[2 * e][j >> 1],
                                                 j & 1 ? 0x07060302u : 0x05040100u);
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[rt][j] = mfma16(a, pf[rt], acc[rt][j]);
        }
    };

    int blk = split * sh.per + wave;
    if (blk < blk_end) {
        KeyRegs<D, I8> kr;
        ValueRegs<D, I8> vr;
        int64_t row[2], next[2];
        rows_of(blk, row);
        load_k(row, kr);
        for (; blk < blk_end; blk += 4) {
            load_v(row, vr);
            KeyRegs<D, I8> kn;
            rows_of(min(blk + 4, blk_end - 1), next);
            load_k(next, kn);
            step(blk, row, kr, vr);
            kr = kn;
            row[0] = next[0], row[1] = next[1];
        }
    }

    // The waves' maxima and sums, then their outputs, joined in wave order.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        l[rt] += __shfl_xor(l[rt], 16, 64);
        l[rt] += __shfl_xor(l[rt], 32, 64);
        if (quad == 0) {
            s_m[wave][16 * rt + c] = m[rt];
            s_l[wave][16 * rt + c] = l[rt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (r0 + 16 * rt > last) break;
        float mx = s_m[0][16 * rt + c];
#pragma unroll
        for (int w = 1; w < 4; ++w) mx = fmaxf(mx, s_m[w][16 * rt + c]);
        const float f = m[rt] == kNone ? (l[rt] == l[rt] ? 0.f : 1.f) : exp2_fast(m[rt] - mx);
        if (rt) __syncthreads();
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s_o[wave][c * kRowPad + (4 * quad + i) * kCols + j] = acc[rt][j][i] * f;
        __syncthreads();
        // 16 threads a row, D / 16 columns each
        const int row = threadIdx.x >> 4, col = (threadIdx.x & 15) * kCols;
        const int r = r0 + 16 * rt + row;
        if (r <= last) {
            float o[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                o[j] = s_o[0][row * kRowPad + col + j];
#pragma unroll
                for (int w = 1; w < 4; ++w) o[j] += s_o[w][row * kRowPad + col + j];
            }
            float M = s_m[0][16 * rt + row], L = 0.f;
#pragma unroll
            for (int w = 1; w < 4; ++w) M = fmaxf(M, s_m[w][16 * rt + row]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float mw = s_m[w][16 * rt + row], lw = s_l[w][16 * rt + row];
                L += lw * (mw == kNone ? 1.f : exp2_fast(mw - M));  // no maximum: the sum is 0 or NaN
            }
            const int i = r / p.G;
            const int64_t at = (int64_t)(sq.start + i) * p.Hq + h * p.G + (r - i * p.G);
            if (sh.used == 1) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                uint32_t v[kCols / 2];
#pragma unroll
                for (int j = 0; j < kCols / 2; ++j) v[j] = pack_bf16(o[2 * j] * inv, o[2 * j + 1] * inv);
                uint32_t *dst = (uint32_t *)(p.out + at * D + col);
#pragma unroll
                for (int j = 0; j < kCols / 2; ++j) dst[j] = v[j];
            } else {
                const int64_t pr = (int64_t)split * p.T * p.Hq + at;
                float *dst = p.part + pr * D + col;
#pragma unroll
                for (int j = 0; j < kCols; ++j) dst[j] = o[j];
                if ((threadIdx.x & 15) == 0) {
                    p.part_ml[pr * 2] = M;
                    p.part_ml[pr * 2 + 1] = L;
                }
            }
        }
    }
}

// Joins the splits of a row, in split order: one wave a row, D / 64 columns a lane.
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnParams p, int block_rows, int waves)
{
    constexpr int kPer = D / 64;
    const int lane = threadIdx.x & 63;
    const int b = blockIdx.y;
    const Seq sq = seq_of(p, b);
    const int64_t x = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int i = (int)(x / p.Hq), hq = (int)(x - (int64_t)i * p.Hq);
    if (i >= sq.n) return;
    const int r = i * p.G + hq % p.G;
    const int last = min(sq.n * p.G, (r / block_rows + 1) * block_rows) - 1;
    const Share sh = share_of(tokens_of(sq, last, p.G), p.splits, waves);
    if (sh.used == 1) return;
    const int64_t at = (int64_t)(sq.start + i) * p.Hq + hq, stride = (int64_t)p.T * p.Hq;
    float M = kNone, L = 0.f, o[kPer] = {};
    for (int s = 0; s < sh.used; ++s) M = fmaxf(M, p.part_ml[(s * stride + at) * 2]);
#pragma unroll 4
    for (int s = 0; s < sh.used; ++s) {
        const float *ml = p.part_ml + (s * stride + at) * 2;
        const float f = ml[0] == kNone ? 1.f : exp2_fast(ml[0] - M);  // no maximum: zeros or NaN
        L += ml[1] * f;
        const float *src = p.part + (s * stride + at) * D + lane * kPer;
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[j] += src[j] * f;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if constexpr (kPer == 2)
        ((uint32_t *)(p.out + at * D))[lane] = pack_bf16(o[0] * inv, o[1] * inv);
    else
        ((__bf16 *)(p.out + at * D))[lane] = (__bf16)(o[0] * inv);
}

template <int D, bool I8, int RT>
void launch_rows(const AttnParams &p, int64_t B, int64_t max_rows, hipStream_t stream)
{
    const dim3 grid((unsigned)((max_rows + 16 * RT - 1) / (16 * RT) * p.splits), (unsigned)p.Hkv, (unsigned)B);
    hipLaunchKernelGGL((attn_rows_kernel<D, I8, RT>), grid, dim3(256), 0, stream, p);
}

template <int D, bool I8>
void launch_attention(const AttnParams &p, int64_t B, int64_t max_q, int rt, hipStream_t stream)
{
    const int64_t max_rows = max_q * p.G;
    switch (rt) {
    case 1: launch_rows<D, I8, 1>(p, B, max_rows, stream); break;
    case 2: launch_rows<D, I8, 2>(p, B, max_rows, stream); break;
    case 3: launch_rows<D, I8, 3>(p, B, max_rows, stream); break;
    default: launch_rows<D, I8, 4>(p, B, max_rows, stream); break;
    }
    if (p.splits > 1) {
        const dim3 grid((unsigned)((max_q * p.Hq + 3) / 4), (unsigned)B);
        hipLaunchKernelGGL(attn_join_kernel<D>, grid, dim3(256), 0, stream, p, 16 * rt, 4);
    }
}

}  // namespace

extern "C" {

w4_status w4_paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, const void *k_cache,
                             const void *v_cache, const float *k_scale, const float *v_scale, int cache_bits,
                             const int32_t *block_table, int64_t table_stride, int64_t table_width,
                             const int32_t *q_start, const int32_t *kv_len, void *out, float scale, int64_t T,
                             int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t pages,
                             int64_t page_size, int64_t max_q, int64_t max_kv, void *stream)
{
    if (cache_bits != 16 && cache_bits != 8) {
        set_error("w4_paged_attention: cache_bits=%d: need 16 or 8", cache_bits);
        return W4_ERR_SHAPE;
    }
    if (D != 64 && D != 128) {
        set_error("w4_paged_attention: D=%lld: need 64 or 128", (long long)D);
        return W4_ERR_SHAPE;
    }
    if (T < 0 || B < 0 || B > 65535 || kv_heads < 1 || kv_heads > 65535 || q_heads < kv_heads ||
        q_heads % kv_heads != 0 || q_heads > 65536 || T > 0x7FFFFFFF / q_heads) {
        set_error("w4_paged_attention: T=%lld B=%lld q_heads=%lld kv_heads=%lld: need 0<=B<=65535, q_heads a multiple "
                  "of kv_heads, T*q_heads<2^31", (long long)T, (long long)B, (long long)q_heads, (long long)kv_heads);
        return W4_ERR_SHAPE;
    }
    if (pages < 1 || page_size < 16 || page_size > 4096 || page_size % 16 != 0 || pages > 0x7FFFFFFF ||
        pages > ((int64_t)1 << 40) / (kv_heads * page_size * D)) {
        set_error("w4_paged_attention: pages=%lld page_size=%lld: need page_size a multiple of 16 up to 4096",
                  (long long)pages, (long long)page_size);
        return W4_ERR_SHAPE;
    }
    const int64_t lim = (int64_t)1 << 32;
    if (table_width < 0 || table_width > 0x7FFFFFFF || table_stride < table_width || table_stride > lim || max_q < 0 ||
        max_q > T || max_kv < 0 || max_kv > 0x7FFFFFFF || q_token_stride < 0 || q_token_stride > lim ||
        q_head_stride < 0 || q_head_stride > lim) {
        set_error("w4_paged_attention: max_q=%lld max_kv=%lld table_width=%lld, or a stride, is out of range "
                  "(0<=max_q<=T)", (long long)max_q, (long long)max_kv, (long long)table_width);
        return W4_ERR_SHAPE;
    }
    if (T == 0 || B == 0 || max_q == 0) return W4_OK;
    if (!q || !k_cache || !v_cache || !q_start || !kv_len || !out || (table_width > 0 && !block_table) ||
        (cache_bits == 8 && (!k_scale || !v_scale))) {
        set_error("w4_paged_attention: a required pointer is NULL");
        return W4_ERR_NULL;
    }
    if (!aligned(q, 2) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(q_start, 4) || !aligned(kv_len, 4) ||
        (cache_bits == 8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16)))) {
        set_error("w4_paged_attention: the caches, their scales and out must be 16-byte aligned, q 2-byte, the index "
                  "arrays 4-byte");
        return W4_ERR_ALIGN;
    }
    int dev = -1;
    w4_status st = check_device(&dev);
    if (st != W4_OK) return st;
    AttnParams p;
    p.q = (const uint16_t *)q, p.q_tok_stride = q_token_stride, p.q_head_stride = q_head_stride;
    p.k = k_cache, p.v = v_cache, p.ks = k_scale, p.vs = v_scale;
    p.table = block_table, p.table_stride = table_stride, p.q_start = q_start, p.kv_len = kv_len;
    p.out = (uint16_t *)out, p.scale2 = scale * 1.4426950408889634f;
    p.Hq = (int)q_heads, p.Hkv = (int)kv_heads, p.G = (int)(q_heads / kv_heads), p.T = (int)T;
    p.width = (int)table_width, p.pages = (int)pages, p.page_tiles = (int)(page_size / 16);
    p.page_magic = (((uint64_t)1 << 32) + p.page_tiles - 1) / p.page_tiles;
    p.q_vec = aligned(q, 16) && q_token_stride % 8 == 0 && q_head_stride % 8 == 0;
    const int64_t max_rows = max_q * p.G;
    const int rt = max_rows >= 64 ? 4 : (int)((max_rows + 15) / 16);
    const int64_t row_blocks = (max_rows + 16 * rt - 1) / (16 * rt);
    // enough workgroups to fill the card, each wave with one step or more
    const int64_t units = row_blocks * kv_heads * B, steps = (max_kv + 4 * kBlock - 1) / (4 * kBlock);
    int64_t splits = units >= 512 ? 1 : (512 + units - 1) / units;
    if (splits > steps) splits = steps;
    if (splits > 128) splits = 128;
    if (splits < 1) splits = 1;
    p.splits = (int)splits;
    p.part = p.part_ml = nullptr;
    if (splits > 1) {
        unsigned *count = nullptr;
        float *part = nullptr;
        const size_t part_rows = (size_t)splits * T * q_heads;
        st = get_workspace(dev, (hipStream_t)stream, 0, part_rows * (D + 2) * sizeof(float), &count, &part);
        if (st != W4_OK) return st;
        p.part = part, p.part_ml = part + part_rows * D;
    }
    if (row_blocks * splits > 0x7FFFFFFF || max_q * q_heads > 0x7FFFFFFF) {
        set_error("w4_paged_attention: max_q=%lld is too large", (long long)max_q);
        return W4_ERR_SHAPE;
    }
    if (D == 128)
        cache_bits == 8 ? launch_attention<128, true>(p, B, max_q, rt, (hipStream_t)stream)
                        : launch_attention<128, false>(p, B, max_q, rt, (hipStream_t)stream);
    else
        cache_bits == 8 ? launch_attention<64, true>(p, B, max_q, rt, (hipStream_t)stream)
                        : launch_attention<64, false>(p, B, max_q, rt, (hipStream_t)stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail("w4_paged_attention launch", e);
    return W4_OK;
}

}  // extern "C"

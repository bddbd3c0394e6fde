// Attention of single tokens over the 8-bit key/value cache.
//
// For query head q of sequence b (key/value head h = q / G):
//   x_t = scale * (sK/127) * sum_d Q[d] Kc[t,d]          t < len
//   O   = sum_t e^(x_t - max x) * (sV/127) * Vc[t,:] / sum_t e^(x_t - max x)
// in one pass over the codes with a running maximum and sum.
//
// Bound by reading the codes from HBM once (2 D bytes a token and head), so the
// work is cut by bytes: an item is one (sequence, key/value head, tile of up to
// 8*NT queries), the blocks of 64 tokens of all items in order are dealt to the warps
// of a persistent grid in equal contiguous ranges, and every warp works through its
// range alone.  Ranges usually begin and end inside an item; those pieces are merged
// per CTA in shared memory, and the few items that cross CTAs by
// attention_combine_kernel from at most two pieces a CTA, always in the same order.
//
// The codes travel by cp.async into the warp's own slots, four sub-tiles of 16
// tokens: as K's are read, V's are asked for, and as V's are read, the next
// block's K.  With 12 warps that is 48 to 96 KB on the way to every SM.  A lane's
// bytes are its own mma.sync fragments: m16n8k16 with tokens (then V's columns) as
// the 16 rows and queries as the 8 columns, which suits one to eight queries per
// head; at one MMA in ten cycles the legacy tensor path is nowhere near a limit.  (With
// two columns of queries the accumulators fill the registers and leave two warps a
// scheduler.  A tcgen05 product of 128 tokens, or 128 columns of V, by 16 queries would
// keep them in tensor memory; it has not been built.)
//
// Measured: 16 sequences of 2048 tokens, 96 heads of 128: 149 us (805 MB, 5.4 TB/s,
// 82 % of a copy's rate); 16 of 0 to 2048, 15000 tokens in all: 79 us (4.7 TB/s: about
// ten of them are the start, the joins and the uneven end); 64 long ones, 12 queries a
// head: 267 us (4.3 TB/s, bound by instructions); one of 1000 tokens, 40 heads: 14 us.
//
// What counts besides bytes is instructions, most of them to turn codes into fp16:
// xor 0x80 and a byte permute against 0x64 make 1024 + (code + 128), exactly, and a
// subtraction takes the 1152 off again.  (Left in K's operand and taken off the sums
// instead, it costs fp32 sums of the size of 1152 |sum(Q)|: scores that are 0.001 to
// 0.003 off where the queries' mean is 3 to 8, and saves little: 143 us for 149 and 263
// for 267 on the first and third of the calls above.)  p = 2^14 e^(x - max) is rounded
// to fp16 for the second product (2^-11, as the output will be), and the softmax's sum is
// that of the rounded p (one more MMA, with ones for V).  With 2^14 in front a weight
// down to 2^-28 of the largest is a normal number and is rounded by 2^-39 of the largest
// below that: with the largest at 1, weights below 2^-25 were lost, 131072 of which are
// 0.4 % of the result.  The sums over V are kept in units of the current block's scale,
// so the MMAs accumulate in place.
#pragma once

#include "device_common.cuh"
#include "kv_cache.cuh"

namespace i8r {
namespace attn {

constexpr int STEP = 16;                 // tokens per sub-tile (an MMA's rows, or its depth)
constexpr int SUBS = kv::BLOCK / STEP;   // sub-tiles per block
constexpr int DEC_MAX_CTAS = 160;        // of the persistent grid (one per SM), which sizes the workspace

// What attention_combine_kernel needs to know about a CTA: whether it had work, and
// the item that begins in it and ends in another (b < 0: none), with the slot of its
// piece there and the CTA where it ends.
struct Join {
    int b, h, gt, slot, last, worked;
};

struct DecodeParams {
    kv::Cache c;
    const __half *Q;
    __half *O;
    long long ldq, ldo;
    const int32_t *lengths;
    int B, G, GT, tile;                  // queries per kv head, tiles of `tile` queries per kv head
    float scale_log2;                    // |scale| * log2(e)
    uint32_t negate;                     // sign bits that the queries are flipped by: scale < 0
    float *part;                         // [2 * CTAs][tile][D + 2]: pieces that cross CTAs
    float *firsts;                       // [warps of the grid][tile][D + 2]: warps' first pieces (wide tiles)
    Join *joins;                         // [CTAs]
};

// Floats of one piece: maximum, sum and D values per query.
__host__ __device__ constexpr int piece_floats(int tile, int D) { return tile * (D + 2); }
// Bytes of one warp's slots: four sub-tiles, K's and V's in turn, or (two columns of
// queries: fewer warps) eight, four for each.  In the end its last piece.
__host__ __device__ constexpr int ring_bytes(int tile, int D) { return (tile > 8 ? 2 : 1) * kv::BLOCK * D; }
// Bytes of one warp's queries, in the order of their MMA fragments.
__host__ __device__ constexpr int query_bytes(int tile, int D) { return D / 16 * (tile > 8 ? 2 : 1) * 256; }
__host__ __device__ constexpr size_t decode_smem(int tile, int D, int warps) {
    return static_cast<size_t>(warps) *
           (ring_bytes(tile, D) + query_bytes(tile, D) + (tile > 8 ? 0 : piece_floats(tile, D) * 4));
}
// Warps per CTA, one CTA an SM: 12 of 168 registers a lane, or with two columns of
// queries 8 of 255 (12, with the queries' fragments read from shared memory for
// every 32 tokens, were slower: 289 us for 269 on 64 long sequences of 12 queries a head).
__host__ __device__ constexpr int dec_warps(int nt) { return nt == 1 ? 12 : 8; }
constexpr size_t DEC_SMEM = 226 * 1024;
static_assert(decode_smem(8, 128, dec_warps(1)) <= DEC_SMEM && decode_smem(16, 128, dec_warps(2)) <= DEC_SMEM, "the widest tiles fit");
static_assert(piece_floats(8, 64) * 4 <= ring_bytes(8, 64) && piece_floats(16, 64) * 4 <= ring_bytes(16, 64) &&
              piece_floats(8, 128) * 4 <= ring_bytes(8, 128) && piece_floats(16, 128) * 4 <= ring_bytes(16, 128),
              "a piece fits a warp's slots");

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// 8-byte asynchronous copy global -> shared; zeros instead with src_bytes = 0.
__device__ __forceinline__ void cp_async_8(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two weights in fp16, a in the low half.  Above fp16's largest value they become that (from
// 2^25 on, a score's rounding exceeds the factor 4 that is left); a NaN stays.
__device__ __forceinline__ uint32_t weights2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
constexpr float DECODE_RAISED = 14.0f;          // log2 of what stands in front of the weights
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two codes as fp16: their bytes of x = codes ^ 0x80 are picked into the low bytes
// of 0x6400, 1024 + byte, which is 1152 more than the code.
template <int kSel>
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
    const uint32_t u = __byte_perm(x, 0x64646464u, kSel);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(1152.0f));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A sequence's length; one out of range (reported) counts as empty.
__device__ __forceinline__ int length_of(const DecodeParams &p, int b) {
    const int n = p.lengths[b];
    if (n < 0 || n > static_cast<long long>(p.c.max_blocks) * kv::BLOCK) {
        report_status(I8R_DEV_BAD_INDEX);
        return 0;
    }
    return n;
}
// Blocks of one item of a sequence of n tokens.
__device__ __forceinline__ int item_blocks(int n) { return (n + kv::BLOCK - 1) / kv::BLOCK; }

// What a warp works on next: a block of the item (sequence b, key/value head h,
// query tile gt).
struct Place {
    int b, h, gt, block, blocks, len;
    // the block after this one; only called while the range has one
    __device__ __forceinline__ void next(const DecodeParams &p) {
        if (++block < blocks) return;
        block = 0;
        if (++gt < p.GT) return;
        gt = 0;
        if (++h < p.c.H) return;
        h = 0;
        do {
            if (++b >= p.B) return;
            len = length_of(p, b);
        } while (len == 0);
        blocks = item_blocks(len);
    }
};

// Where the blocks of all items lie: sequence b's begin after those of the
// sequences before it, H * GT items of item_blocks(len) each.  A lane keeps four
// sequences' lengths of the first 128, which is all of them in most calls; more
// are read again where they are needed.  Ranges are cut between blocks: a warp
// takes about as long for a part of one.
struct Order {
    int len[4];
    long long before;                    // blocks of the sequences before this lane's four
    long long total;
    int warps;                           // of the grid
    long long share;                     // blocks of a warp, and what is left over
    int rest;

    __device__ __forceinline__ static void lengths(const DecodeParams &p, int b0, int (&n)[4]) {
        const int b = b0 + 4 * (threadIdx.x & 31);
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = b + j < p.B ? length_of(p, b + j) : 0;
    }
    __device__ __forceinline__ static long long blocks_of(const DecodeParams &p, const int (&n)[4]) {
        return (static_cast<long long>(item_blocks(n[0])) + item_blocks(n[1]) + item_blocks(n[2]) + item_blocks(n[3])) *
               (p.c.H * p.GT);
    }
    __device__ __forceinline__ static long long scan(const DecodeParams &p, const int (&n)[4], long long *prior) {
        const int lane = threadIdx.x & 31;
        const long long mine = blocks_of(p, n);
        long long sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += up;
        }
        *prior = sum - mine;
        return __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    __device__ __forceinline__ void load(const DecodeParams &p, int grid_warps) {
        warps = grid_warps;
        lengths(p, 0, len);
        total = scan(p, len, &before);
        for (int b0 = 128; b0 < p.B; b0 += 128) {
            int n[4];
            long long prior;
            lengths(p, b0, n);
            total += scan(p, n, &prior);
        }
        share = total / warps;
        rest = static_cast<int>(total - share * warps);
    }
    // The first block of warp w's range, floor(total * w / warps), and the warp whose range holds
    // block u < total (so total > 0).
    __device__ __forceinline__ long long begin(int w) const {
        return share * w + static_cast<unsigned>(rest * w) / static_cast<unsigned>(warps);
    }
    __device__ __forceinline__ static int owner(long long u, int warps, long long total) {
        return static_cast<int>(((u + 1) * warps - 1) / total);
    }
    // Block u < total.
    __device__ __forceinline__ void find(const DecodeParams &p, long long u, Place *w) const {
        const int lane = threadIdx.x & 31;
        int v[4] = {len[0], len[1], len[2], len[3]};
        long long prior = before, base = 0;
        for (int b0 = 0; b0 < p.B; b0 += 128) {
            if (b0) {
                lengths(p, b0, v);
                scan(p, v, &prior);
            }
            const long long mine = blocks_of(p, v);
            long long r = u - base - prior;                          // within this lane's four sequences
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, r >= 0 && r < mine);
            if (hit) {
                const int at = __ffs(hit) - 1;
                int k = 0;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const long long c = static_cast<long long>(item_blocks(v[j])) * (p.c.H * p.GT);
                    if (k == j && r >= c) r -= c, k = j + 1;
                }
                const int own = k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3];
                // within one sequence: H * GT * max_blocks at most, which the host checks
                const unsigned in = static_cast<unsigned>(__shfl_sync(0xFFFFFFFFu, r, at));
                w->len = __shfl_sync(0xFFFFFFFFu, own, at);
                w->b = __shfl_sync(0xFFFFFFFFu, b0 + 4 * lane + k, at);
                w->blocks = item_blocks(w->len);
                const unsigned hg = in / static_cast<unsigned>(w->blocks);
                w->block = static_cast<int>(in - hg * w->blocks);
                w->h = static_cast<int>(hg / p.GT);
                w->gt = static_cast<int>(hg % p.GT);
                return;
            }
            base += __shfl_sync(0xFFFFFFFFu, prior + mine, 31);
        }
    }
};

// A window of 32 of a sequence's block numbers, one a lane: the table is read once
// per 32 blocks (and serves all heads of a shorter sequence), not in front of every
// block's codes.
struct Window {
    int b = -1, first = 0, mine = 0;
    // where a place's block and head lie, in blocks of one head (the host checks that
    // 32 bits hold them); a bad block number (reported) reads block 0, which is always there
    __device__ __forceinline__ uint32_t slot(const DecodeParams &p, const Place &w) {
        const int i = w.block;
        if (w.b != b || i < first || i >= first + 32) {
            b = w.b;
            first = i & ~31;
            const int at = first + (threadIdx.x & 31);
            mine = at < p.c.max_blocks ? p.c.table[static_cast<size_t>(b) * p.c.max_blocks + at] : -1;
        }
        int page = __shfl_sync(0xFFFFFFFFu, mine, i - first);
        if (page < 0 || page >= p.c.num_blocks) {
            report_status(I8R_DEV_BAD_INDEX);
            page = 0;
        }
        return static_cast<uint32_t>(page) * p.c.H + w.h;
    }
};

template <int D>
__device__ __forceinline__ const int8_t *block_codes(const int8_t *codes, uint32_t slot) {
    return codes + static_cast<size_t>(slot) * (kv::BLOCK * D);
}

// Sub-tile j (16 tokens) of K: this lane's own bytes of it, in the order in which
// it reads them back: rows (tokens) g and g + 8, 16 bytes at 16t of each 64.  Four
// neighbouring lanes cover 64 bytes of a row.
template <int D>
__device__ __forceinline__ void issue_k(const int8_t *K, int j, uint32_t ring) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int8_t *src = K + (STEP * j + g) * D + 16 * t;
    uint32_t dst = ring + j * (STEP * D) + lane * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < D / 64; ++c, dst += 512) cp_async_16(dst, src + 8 * r * D + 64 * c, 16u);
}

// Sub-tile j of V: a lane reads rows 2t, 2t+1, 2t+8, 2t+9, the D/8 bytes at g*D/8 of
// each, which for neighbouring lanes lie in different rows.  Copied that way, every
// 32 bytes were a request of their own (three times the L1's requests and half as
// many sectors again: 4.6 TB/s without any arithmetic, for 6.3 in whole rows); so
// the lanes copy whole rows for one another.  Row r's bytes are at v_row(r), its
// 16-byte pieces swapped by v_swap(r), which keeps both the copies' and the
// reads' eight lanes on different banks.
template <int D>
__device__ __forceinline__ int v_row(int r) {
    // D = 128: the four rows of one MMA register (t = 0..3) side by side; D = 64: even
    // and odd t in the two halves of 128 bytes
    const int t = (r >> 1) & 3, k = (r & 1) + 2 * (r >> 3);
    return (4 * k + t) * D;
}
template <int D>
__device__ __forceinline__ int v_swap(int r) {
    const int t = (r >> 1) & 3;
    return D == 128 ? 2 * t : 2 * (t >> 1);
}
template <int D>
__device__ __forceinline__ void issue_v(const int8_t *V, int j, uint32_t ring) {
    constexpr int PIECES = D / 16, ROWS = 32 / PIECES;          // 16-byte pieces of a row, rows per instruction
    const int lane = threadIdx.x & 31, piece = lane % PIECES;
#pragma unroll
    for (int i = 0; i < STEP / ROWS; ++i) {
        const int r = i * ROWS + lane / PIECES;
        cp_async_16(ring + j * (STEP * D) + v_row<D>(r) + ((piece ^ v_swap<D>(r)) << 4),
                    V + (STEP * j + r) * D + 16 * piece, 16u);
    }
}

// The queries of an item, this lane's own fragments: for each 16 values of D and 8
// queries, values 16t + 64 (k/4) + 4 (k%4) .. + 3 of query g (zeros past the last one).
template <int D, int NT>
__device__ __forceinline__ void issue_q(const DecodeParams &p, const Place &w, uint32_t queries) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int q0 = w.gt * p.tile;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int qi = 8 * n + g;
        const bool have = q0 + qi < p.G && qi < p.tile;
        const __half *src = p.Q + static_cast<size_t>(w.b) * p.ldq;
        if (have) src += static_cast<size_t>(w.h * p.G + q0 + qi) * D + 16 * t;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            cp_async_8(queries + (k * NT + n) * 256 + lane * 8, have ? src + 64 * (k >> 2) + 4 * (k & 3) : src, have ? 8u : 0u);
    }
}

// One piece of an item in memory: per query its maximum - DECODE_RAISED (log2 units), its sum
// and its D unnormalised values.
template <int D>
__device__ __forceinline__ float *piece_row(float *piece, int q) { return piece + q * (D + 2); }

template <int D, int NT>
struct State {
    float acc[D / 16][NT][4];            // in units of vs
    float m[NT][2], l[NT][2];            // maximum - DECODE_RAISED (log2 units) and sum of this lane's queries 2t, 2t + 1: the same in all its g
    float vs;                            // the scale acc is in (sV/127 of the last block with any)
    uint2 q[D / 16][NT];                 // the queries' fragments

    // a new item: nothing summed yet
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
        vs = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][n][e] = 0.0f;
    }

    // its queries, once they have come
    __device__ __forceinline__ void take_queries(const DecodeParams &p, const uint8_t *queries) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint2 v = reinterpret_cast<const uint2 *>(queries + (k * NT + n) * 256)[lane];
                v.x ^= p.negate;
                v.y ^= p.negate;
                q[k][n] = v;
            }
    }

    // Scores of sub-tiles j and j + 1: rows are tokens g and g+8, a lane's four
    // codes of a word are the MMA's columns 2t, 2t+1, 2t+8, 2t+9 (so are the
    // queries').  Four chains of MMAs go side by side (two sub-tiles, and two halves
    // of each sum or two columns of queries): a chain alone waits for each MMA's result.
    __device__ __forceinline__ void scores(const uint8_t *ring, int j, float (&x)[2][NT][4]) const {
        float y[2][NT][4];
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[s][n][e] = y[s][n][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint32_t a[2][4], b[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint8_t *mine = ring + (j + s) * (STEP * D) + lane * 16;
                const uint4 r0 = *reinterpret_cast<const uint4 *>(mine + 512 * c);
                const uint4 r1 = *reinterpret_cast<const uint4 *>(mine + 512 * (D / 64 + c));
                a[s][0] = r0.x, a[s][1] = r0.y, a[s][2] = r0.z, a[s][3] = r0.w;
                b[s][0] = r1.x, b[s][1] = r1.y, b[s][2] = r1.z, b[s][3] = r1.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t u = a[s][k] ^ 0x80808080u, v = b[s][k] ^ 0x80808080u;
                    const uint32_t a0 = code_pair<0x4140>(u), a2 = code_pair<0x4342>(u);
                    const uint32_t a1 = code_pair<0x4140>(v), a3 = code_pair<0x4342>(v);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816(NT == 1 && (k & 1) ? y[s][n] : x[s][n], a0, a1, a2, a3, q[4 * c + k][n].x, q[4 * c + k][n].y);
                }
            }
        }
        if (NT == 1) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[s][0][e] += y[s][0][e];
        }
    }

    // The block's scores become weights (in `pf`, as the second product's
    // fragments), the maxima and sums move on, and acc is rescaled to them and to
    // the block's V scale.  Tokens from hi on weigh nothing.
    __device__ __forceinline__ void weigh(const DecodeParams &p, float (&x)[SUBS / 2][2][NT][4], float sk, float sv, int hi,
                                          uint32_t (&pf)[SUBS][NT][2]) {
        const int g = (threadIdx.x & 31) >> 2;
        // s/127 as a product (2^-24 more than the division); an infinite sK makes every score NaN, not
        // only those of codes whose sum is not negative: a code of 0 stands for NaN then
        const float ks = fmaf(sk, 0.0f, p.scale_log2 * (sk * (1.0f / 127.0f))), now = sv * (1.0f / 127.0f);
        // a block whose scale is 0 stands for zeros, whatever its codes: values() is not called for it
        const bool nothing = now == 0.0f;
        const float turn = nothing ? 1.0f : vs / now;
        if (!nothing) vs = now;
        const bool cut = hi < kv::BLOCK;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float keep[2], alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < SUBS; ++j) {
                    float &u = x[j >> 1][j & 1][n][e], &v = x[j >> 1][j & 1][n][2 + e];
                    if (cut) {
                        const int t0 = STEP * j + g;
                        u = t0 < hi ? u : -INFINITY;
                        v = t0 + 8 < hi ? v : -INFINITY;
                    }
                    top = fmaxf(top, fmaxf(u, v));
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                const float to = fmaxf(fmaf(top, ks, -DECODE_RAISED), m[n][e]);
                alpha[e] = ex2(m[n][e] - to);
                m[n][e] = to;
#pragma unroll
                for (int j = 0; j < SUBS; ++j) {
                    float &u = x[j >> 1][j & 1][n][e], &v = x[j >> 1][j & 1][n][2 + e];
                    const bool in0 = !cut || u != -INFINITY, in1 = !cut || v != -INFINITY;
                    u = in0 ? ex2(fmaf(u, ks, -to)) : 0.0f;
                    v = in1 ? ex2(fmaf(v, ks, -to)) : 0.0f;
                }
                keep[e] = alpha[e] * turn;
            }
            // the weights' sum over the block's tokens, the same in every row of the MMA's result
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            constexpr uint32_t kOnes = 0x3C003C00u;
#pragma unroll
            for (int j = 0; j < SUBS; ++j) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    pf[j][n][r] = transpose8x8(weights2(x[j >> 1][j & 1][n][2 * r], x[j >> 1][j & 1][n][2 * r + 1]));
                mma16816(sum, kOnes, kOnes, kOnes, kOnes, pf[j][n][0], pf[j][n][1]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) l[n][e] = fmaf(l[n][e], alpha[e], sum[e]);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][n][e] *= keep[e & 1];
        }
    }

    // Sub-tile j's values: rows are columns d of V, two per lane and MMA; k is the token.
    __device__ __forceinline__ void values(const uint8_t *ring, int j, const uint32_t (&pf)[NT][2]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        uint32_t v[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 2 * t + (k & 1) + 8 * (k >> 1);
            const uint8_t *mine = ring + j * (STEP * D) + v_row<D>(r);
            if (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4 *>(mine + ((g ^ v_swap<D>(r)) << 4));
                v[k][0] = w.x, v[k][1] = w.y, v[k][D / 32 - 2] = w.z, v[k][D / 32 - 1] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(mine + (((g >> 1) ^ v_swap<D>(r)) << 4) + 8 * (g & 1));
                v[k][0] = w.x, v[k][1] = w.y;
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k][i] ^= 0x80808080u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t lo = half ? __byte_perm(v[0][i], v[1][i], 0x7362) : __byte_perm(v[0][i], v[1][i], 0x5140);
                const uint32_t hi = half ? __byte_perm(v[2][i], v[3][i], 0x7362) : __byte_perm(v[2][i], v[3][i], 0x5140);
                const uint32_t a0 = code_pair<0x4140>(lo), a1 = code_pair<0x4342>(lo);
                const uint32_t a2 = code_pair<0x4140>(hi), a3 = code_pair<0x4342>(hi);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(acc[2 * i + half][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
            }
        }
    }

    // The item's output, or its piece.
    __device__ __forceinline__ void end(const DecodeParams &p, const Place &w, bool whole, float *piece) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int h = w.h, q0 = w.gt * p.tile;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float sum = l[n][e];
                const int qi = 8 * n + 2 * t + e;
                if (qi >= p.tile || q0 + qi >= p.G) continue;
                if (whole) {
                    const float f = vs / sum;
                    __half2 o[D / 16];
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) o[k] = __floats2half2_rn(acc[k][n][e] * f, acc[k][n][2 + e] * f);
                    __half *dst = p.O + static_cast<size_t>(w.b) * p.ldo + static_cast<size_t>(h * p.G + q0 + qi) * D +
                                  g * (D / 8);
#pragma unroll
                    for (int k = 0; k < D / 64; ++k)
                        *reinterpret_cast<uint4 *>(dst + 8 * k) = *reinterpret_cast<const uint4 *>(o + 4 * k);
                } else {
                    float *row = piece_row<D>(piece, qi);
                    if (g == 0) {
                        row[0] = m[n][e];
                        row[1] = sum;
                    }
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        *reinterpret_cast<float2 *>(row + 2 + g * (D / 8) + 2 * k) =
                            make_float2(acc[k][n][e] * vs, acc[k][n][2 + e] * vs);
                }
            }
    }
};

// What a warp left of an item it did not do alone.
struct Piece {
    int b, h, gt;                        // b < 0: none
    bool starts;                         // the piece holds the item's first block
    bool front;                          // it begins where the CTA's range begins
    int left;                            // blocks of the item after it
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * dec_warps(NT), 1)
    attention_decode_kernel(const __grid_constant__ DecodeParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Piece pieces[2 * dec_warps(NT)];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int cta_warps = dec_warps(NT);
    const int warp_ring = ring_bytes(p.tile, D);
    uint8_t *ring = smem + warp * warp_ring;
    // V's slots: K's own, filled in turn, or four more (kSplit)
    constexpr bool kSplit = NT == 2;
    constexpr int kAhead = kSplit ? SUBS - 1 : 1;        // groups of two sub-tiles that may be on the way at a wait
    const uint32_t ring_u = smem_u32(ring), ring_v = ring_u + (kSplit ? SUBS * STEP * D : 0);
    const uint8_t *v_slots = ring + (kSplit ? SUBS * STEP * D : 0);
    uint8_t *queries = smem + cta_warps * warp_ring + warp * query_bytes(p.tile, D);
    const uint32_t queries_u = smem_u32(queries);
    // a warp's first piece is written while its slots are still in use (a wide tile's
    // would take a third of shared memory: it goes to the workspace), its last one into them
    float *firsts = NT == 1 ? reinterpret_cast<float *>(smem + cta_warps * (warp_ring + query_bytes(p.tile, D)))
                            : p.firsts + static_cast<size_t>(blockIdx.x) * cta_warps * piece_floats(p.tile, D);
    if (lane < 2) pieces[2 * warp + lane].b = -1;
    __syncwarp();
    griddep_wait();                      // what the lengths, the cache and the queries come from
    griddep_launch_dependents();         // the combining blocks may take the SMs' places as CTAs leave

    Place w, ahead;
    long long u0, u1, total, cta_end;
    bool front;
    {
        Order order;
        order.load(p, gridDim.x * cta_warps);
        const int me = blockIdx.x * cta_warps + warp;
        u0 = order.begin(me);
        u1 = order.begin(me + 1);
        front = u0 == order.begin(blockIdx.x * cta_warps);
        cta_end = order.begin((blockIdx.x + 1) * cta_warps);
        total = order.total;
        if (u0 < u1) order.find(p, u0, &w);
    }
    if (u0 < u1) {
        int left = static_cast<int>(u1 - u0) - 1;                     // blocks of the range after w
        Window window;
        uint32_t slot = window.slot(p, w), slot_next = 0;
        issue_q<D, NT>(p, w, queries_u);
        {
            const int8_t *K = block_codes<D>(p.c.codes[0], slot);
#pragma unroll
            for (int j = 0; j < SUBS; ++j) {
                issue_k<D>(K, j, ring_u);
                if (j & 1) cp_async_commit();
            }
            if (kSplit) {
                const int8_t *V = block_codes<D>(p.c.codes[1], slot);
#pragma unroll
                for (int j = 0; j < SUBS; ++j) {
                    issue_v<D>(V, j, ring_v);
                    if (j & 1) cp_async_commit();
                }
            }
        }
        float sk = __ldg(p.c.scale[0] + slot), sv = __ldg(p.c.scale[1] + slot);
        State<D, NT> st;
        st.begin();
        ahead = w;
        if (left > 0) {
            ahead.next(p);
            slot_next = window.slot(p, ahead);
        }
        bool starts = w.block == 0, first = true, fresh = true;
        while (true) {
            // the block after this one: its scales now, its codes as the slots come free
            const bool more = left > 0, ends = w.block + 1 == w.blocks;
            float sk_next = 0.0f, sv_next = 0.0f;
            if (more) {
                sk_next = __ldg(p.c.scale[0] + slot_next);
                sv_next = __ldg(p.c.scale[1] + slot_next);
            }
            auto next_k = [&](int j) {
                if (!more) return;
                const int8_t *K = block_codes<D>(p.c.codes[0], slot_next);
                issue_k<D>(K, j, ring_u);
                issue_k<D>(K, j + 1, ring_u);
            };
            auto some_v = [&](int j, uint32_t at) {
                const int8_t *V = block_codes<D>(p.c.codes[1], at);
                issue_v<D>(V, j, ring_v);
                issue_v<D>(V, j + 1, ring_v);
            };
            float x[SUBS / 2][2][NT][4];
#pragma unroll
            for (int j = 0; j < SUBS; j += 2) {
                // a new item's queries came with its first K (kSplit: its last)
                if (kSplit && fresh)
                    cp_async_wait<kAhead - 1>();
                else
                    cp_async_wait<kAhead>();
                if (j == 0 && fresh) st.take_queries(p, queries);
                st.scores(ring, j, x[j / 2]);
                if (kSplit) {
                    if (j + 2 == SUBS && ends && more) issue_q<D, NT>(p, ahead, queries_u);
                    next_k(j);
                } else {
                    __syncwarp();                // read by all: the lanes copy V for one another
                    some_v(j, slot);
                }
                cp_async_commit();
            }
            uint32_t pf[SUBS][NT][2];
            st.weigh(p, x, sk, sv, min(kv::BLOCK, w.len - w.block * kv::BLOCK), pf);
#pragma unroll
            for (int j = 0; j < SUBS; j += 2) {
                cp_async_wait<kAhead>();
                __syncwarp();
                if (sv != 0.0f) {
                    st.values(v_slots, j, pf[j]);
                    st.values(v_slots, j + 1, pf[j + 1]);
                }
                __syncwarp();
                if (kSplit) {
                    if (more) some_v(j, slot_next);
                } else {
                    if (j == 0 && ends && more) issue_q<D, NT>(p, ahead, queries_u);
                    next_k(j);
                }
                cp_async_commit();
            }
            fresh = ends;
            if (ends || !more) {
                const bool whole = starts && ends;
                if (!whole && lane == 0)
                    pieces[2 * warp + (first ? 0 : 1)] = Piece{w.b, w.h, w.gt, starts, first && front, w.blocks - 1 - w.block};
                st.end(p, w, whole, first ? firsts + warp * piece_floats(p.tile, D) : reinterpret_cast<float *>(ring));
                first = false;
                starts = true;
                st.begin();
            }
            if (!more) break;
            w = ahead;
            slot = slot_next;
            sk = sk_next;
            sv = sv_next;
            if (--left > 0) {
                ahead.next(p);
                slot_next = window.slot(p, ahead);
            }
        }
    }
    __syncthreads();

    // Merge this CTA's pieces, item by item in order; an item that begins or ends
    // in another CTA leaves one piece for attention_combine_kernel, in slot 0 if it begins
    // where the CTA's range does, else in slot 1.
    auto piece_of = [&](int k) {
        return (k & 1) ? reinterpret_cast<float *>(smem + (k >> 1) * warp_ring)
                       : firsts + (k >> 1) * piece_floats(p.tile, D);
    };
    bool joined = false;
    for (int i = 0; i < 2 * cta_warps;) {
        const Piece a = pieces[i];
        if (a.b < 0) {
            ++i;
            continue;
        }
        int j = i + 1, last = i;
        for (; j < 2 * cta_warps; ++j) {
            if (pieces[j].b < 0) continue;
            if (pieces[j].b != a.b || pieces[j].h != a.h || pieces[j].gt != a.gt) break;
            last = j;
        }
        const bool whole = a.starts && pieces[last].left == 0;
        const int out_slot = a.front ? 0 : 1;
        // an item that goes on in other CTAs (the last one here, if any)
        if (a.starts && pieces[last].left > 0 && threadIdx.x == 0) {
            const int ends_in = Order::owner(cta_end + pieces[last].left - 1, gridDim.x * cta_warps, total) / cta_warps;
            p.joins[blockIdx.x] = Join{a.b, a.h, a.gt, out_slot, ends_in, 1};
            joined = true;
        }
        float *out = p.part + static_cast<size_t>(2 * blockIdx.x + out_slot) * piece_floats(p.tile, D);
        const int h = a.h, q0 = a.gt * p.tile;
        const int nq = min(p.tile, p.G - q0);
        for (int e = threadIdx.x; e < nq * (D / 2); e += blockDim.x) {
            const int q = e / (D / 2), d = 2 * (e % (D / 2));
            float top = -INFINITY;
            for (int k = i; k <= last; ++k)
                if (pieces[k].b >= 0) top = fmaxf(top, piece_row<D>(piece_of(k), q)[0]);
            float sum = 0.0f;
            float2 o = make_float2(0.0f, 0.0f);
            for (int k = i; k <= last; ++k) {
                if (pieces[k].b < 0) continue;
                const float *row = piece_row<D>(piece_of(k), q);
                const float wgt = ex2(row[0] - top);
                const float2 v = *reinterpret_cast<const float2 *>(row + 2 + d);
                sum = fmaf(wgt, row[1], sum);
                o.x = fmaf(wgt, v.x, o.x);
                o.y = fmaf(wgt, v.y, o.y);
            }
            if (whole) {
                const float inv = 1.0f / sum;
                *reinterpret_cast<__half2 *>(p.O + static_cast<size_t>(a.b) * p.ldo +
                                             static_cast<size_t>(h * p.G + q0 + q) * D + d) =
                    __floats2half2_rn(o.x * inv, o.y * inv);
            } else {
                float *row = piece_row<D>(out, q);
                if (d == 0) {
                    row[0] = top;
                    row[1] = sum;
                }
                *reinterpret_cast<float2 *>(row + 2 + d) = o;
            }
        }
        i = j;
    }
    if (threadIdx.x == 0 && !joined) p.joins[blockIdx.x] = Join{-1, 0, 0, 0, 0, u0 < cta_end ? 1 : 0};
    // sequences without tokens
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (length_of(p, b) == 0)
            for (int i = threadIdx.x; i < p.c.H * p.G * (D / 8); i += blockDim.x)
                *reinterpret_cast<uint4 *>(p.O + static_cast<size_t>(b) * p.ldo + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
}

// The items that cross CTAs.  Block (c, q): query q of the item that begins in CTA
// c's range and ends in a later one's is the sum of the pieces of those CTAs.  One
// thread per value; the pieces are read in order, eight at a time.
template <int D>
__global__ void __launch_bounds__(D) attention_combine_kernel(const __grid_constant__ DecodeParams p) {
    // every block waits, also one without an item: the kernels after this one in the
    // stream wait for this grid alone
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x, q = blockIdx.y, d = threadIdx.x;
    const Join join = p.joins[c];
    const int q0 = join.gt * p.tile;
    if (join.b < 0 || q0 + q >= p.G) return;
    float top = -INFINITY, sum = 0.0f, o = 0.0f;
    for (int k0 = c; k0 <= join.last; k0 += 8) {
        float m[8], l[8], v[8], was = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // in the CTAs after the first it begins where their ranges do; a CTA without
            // blocks (fewer blocks than CTAs) has no piece
            const int cta = k0 + k;
            m[k] = -INFINITY;
            l[k] = v[k] = 0.0f;
            if (cta <= join.last && p.joins[cta].worked) {
                const float *r = piece_row<D>(
                    p.part + static_cast<size_t>(2 * cta + (cta == c ? join.slot : 0)) * piece_floats(p.tile, D), q);
                m[k] = __ldcg(r);
                l[k] = __ldcg(r + 1);
                v[k] = __ldcg(r + 2 + d);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, m[k]);
        const float keep = ex2(was - top);
        sum *= keep;
        o *= keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float wgt = ex2(m[k] - top);
            sum = fmaf(wgt, l[k], sum);
            o = fmaf(wgt, v[k], o);
        }
    }
    p.O[static_cast<size_t>(join.b) * p.ldo + static_cast<size_t>(join.h * p.G + q0 + q) * D + d] = __float2half_rn(o / sum);
}

}  // namespace attn
}  // namespace i8r

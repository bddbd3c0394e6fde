// The 8-bit key/value cache: appending new rows, and reading rows back.
//
// A block is 64 tokens of one sequence.  Per block and key/value head it holds
// 64 x D int8 codes (contiguous, 8 KB at D = 128) and one fp32 absmax scale, the
// library's codec: code = clamp(rhaz(x * fl32(127/scale)), +-127), and a code
// stands for code * scale / 127.  A partly filled block's scale grows with the
// rows it is given: when the new rows' absmax exceeds the old scale, the codes
// already there are rescaled once, code' = rhaz(code * fl32(old/new)).
//
// Both kernels are bound by HBM for prompts: append reads 2 bytes and writes 1
// per value, read-back reads 1 and writes 2.  4096 tokens of 96 heads of 128:
// append 58 us (5.2 TB/s; one warp a block, and the rounding with conversions that
// run at an eighth of the rate, took 123), read-back 56 us (5.4 TB/s).  Single
// tokens are bound by latency: 8 to 10 us for 16 sequences, the chain of finding
// the block, its scale and its rows.
#pragma once

#include "device_common.cuh"

namespace i8r {
namespace kv {

constexpr int BLOCK = 64;            // tokens per cache block
constexpr int WARPS = 8;             // warps per CTA: a (head, K or V) is one's or, appending prompts, four warps'

struct Cache {
    int8_t *codes[2];                // K, V: [num_blocks, H, BLOCK, D]
    float *scale[2];                 // K, V: [num_blocks, H]
    int num_blocks, H, D;
    const int32_t *table;            // [B, max_blocks]
    int max_blocks;
};

// The block number that holds block `i` of sequence b, or -1 (reported) when
// the table has no such entry or it names no block.
__device__ __forceinline__ int block_of(const int32_t *table, int max_blocks, int num_blocks, int b, int i) {
    int page = -1;
    if (i >= 0 && i < max_blocks) page = table[static_cast<size_t>(b) * max_blocks + i];
    if (page < 0 || page >= num_blocks) {
        report_status(I8R_DEV_BAD_INDEX);
        return -1;
    }
    return page;
}

// Which sequence item `item` belongs to, and its place there, when sequence b
// has count(b) items: a warp adds 128 sequences' counts at a time, four
// consecutive ones a lane (their loads are in flight together).  Returns -1
// past the last item.  All lanes get the same answer.  The search begins at
// sequence *from (a multiple of 128), which *before items precede, and leaves both
// where it ended: a search for a later item may go on from there.
template <typename Count>
__device__ __forceinline__ int find_item(long long item, int B, long long *place, Count &&count, int *from, long long *before) {
    const int lane = threadIdx.x & 31;
    long long base = *before;
    for (int b0 = *from; b0 < B; b0 += 128) {
        int n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = b0 + 4 * lane + j < B ? count(b0 + 4 * lane + j) : 0;
        const long long mine = static_cast<long long>(n[0]) + n[1] + n[2] + n[3];
        long long sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += up;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, base + sum > item);
        if (past) {
            long long left = item - base - (sum - mine);
            int j = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (j == k && left >= n[k]) left -= n[k], j = k + 1;
            const int at = __ffs(past) - 1;
            *from = b0;
            *before = base;
            *place = __shfl_sync(0xFFFFFFFFu, left, at);
            return __shfl_sync(0xFFFFFFFFu, b0 + 4 * lane + j, at);
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return -1;
}

template <typename Count>
__device__ __forceinline__ int find_item(long long item, int B, long long *place, Count &&count) {
    int from = 0;
    long long before = 0;
    return find_item(item, B, place, count, &from, &before);
}

// The same by a whole CTA of WARPS warps, 128 sequences a warp at a time; every
// thread of the CTA calls it.  For more than 128 sequences (kMany: append for 4096 of
// one token, 8 heads, 278 -> 94 us); up to there, where each warp has one look, the
// kernels without it are 1 us faster.
template <typename Count>
__device__ __forceinline__ int find_item_cta(long long item, int B, long long *place, Count &&count) {
    __shared__ long long sums[2][WARPS], found_place;
    __shared__ int found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0, turn = 0; b0 < B; b0 += 128 * WARPS, turn ^= 1) {
        const int mine = b0 + 128 * warp + 4 * lane;
        int n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = mine + j < B ? count(mine + j) : 0;
        long long sum = static_cast<long long>(n[0]) + n[1] + n[2] + n[3];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) sums[turn][warp] = sum;
        __syncthreads();
        long long before = base;
        int hit = -1;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (hit < 0 && item < base + sums[turn][w]) hit = w, before = base;
            base += sums[turn][w];
        }
        if (hit >= 0) {
            if (warp == hit) {                                   // this warp's 128 again, to the sequence
                int from = b0 + 128 * warp;
                long long at = 0;
                const int b = find_item(item, B, &at, count, &from, &before);
                if (lane == 0) {
                    found = b;
                    found_place = at;
                }
            }
            __syncthreads();
            *place = found_place;
            return found;
        }
    }
    return -1;
}

// A sequence's row range [lo, hi) in packed rows, from cumulative counts; an
// inconsistent pair (reported) counts as empty.
__device__ __forceinline__ int2 row_range(const int32_t *cu, int b, int rows) {
    const int lo = cu[b], hi = cu[b + 1];
    if (lo < 0 || hi < lo || hi > rows) {
        report_status(I8R_DEV_BAD_INDEX);
        return make_int2(0, 0);
    }
    return make_int2(lo, hi);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Largest magnitude bits of eight fp16 values (a NaN's exceed infinity's, so a
// NaN makes the scale NaN and shows in every value of its block).
__device__ __forceinline__ uint32_t max_bits(const uint4 &v, uint32_t m) {
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// |code| of one value, in bits 8..15 of the result: |x * inv| clamped to 127, plus
// a half, cut to a whole number.  The sum with 2^15 is cut to a multiple of 2^-8,
// towards zero, which never reaches the next whole number; so this is
// round-half-away, without the conversions that run at an eighth of the rate.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
    return __float_as_uint(__fadd_rz(fminf(fabsf(__fmul_rn(x, inv)), 127.0f), 32768.5f));
}

// The codes of four values (two words of fp16 pairs), with the values' signs.
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&w0));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&w1));
    const uint32_t lo = __byte_perm(code_bits(f0.x, inv), code_bits(f0.y, inv), 0x0051);
    const uint32_t hi = __byte_perm(code_bits(f1.x, inv), code_bits(f1.y, inv), 0x0051);
    uint32_t sign;                                 // 0xFF where the value is negative
    asm("prmt.b32 %0, %1, %2, 0xFDB9;" : "=r"(sign) : "r"(w0), "r"(w1));
    // a byte's two's complement: inverted, plus one; no carry leaves its byte
    const uint32_t a = __byte_perm(lo, hi, 0x5410) ^ sign;
    return ((a & 0x7F7F7F7Fu) + (sign & 0x01010101u)) ^ (a & 0x80808080u);
}

__device__ __forceinline__ uint2 codes8(const uint4 &v, float inv) {
    return make_uint2(codes4(v.x, v.y, inv), codes4(v.z, v.w, inv));
}

struct AppendParams {
    Cache c;
    const __half *x[2];              // K, V: new rows, head h of row r at x + r*ld + h*D
    long long ld[2];
    int n_new, B;
    const int32_t *cu_new;           // [B+1]
    const int32_t *past;             // [B]
};

// Blocks that sequence b's new rows touch.
__device__ __forceinline__ int touched_blocks(const AppendParams &p, int b) {
    const int2 r = row_range(p.cu_new, b, p.n_new);
    const int past = p.past[b];
    if (r.x == r.y) return 0;
    if (past < 0 || past > 0x7FFFFFFF - 2 * BLOCK - (r.y - r.x)) {
        report_status(I8R_DEV_BAD_INDEX);
        return 0;
    }
    return (past % BLOCK + (r.y - r.x) + BLOCK - 1) / BLOCK;
}

// kTeam warps per (touched block, head, K or V), each with every kTeam-th
// warp-wide load (256/D rows).  kHold loads a warp stay in registers between the
// absmax and the codes; rows past them are read a second time.  Prompts take
// teams of four that hold a block among them; single tokens one warp that holds
// little, so that more jobs fit an SM.
template <int D, int kHold, int kTeam, bool kMany>
__global__ void __launch_bounds__(32 * WARPS, 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int LANES = D / 8;                   // lanes per row (16 bytes each)
    constexpr int RPL = 32 / LANES;                // rows per warp-wide load
    const int lane = threadIdx.x & 31;
    const int sub = lane / LANES, col = (lane % LANES) * 8;
    const int team = (threadIdx.x >> 5) / kTeam, part = (threadIdx.x >> 5) % kTeam;
    const int first = part * RPL + sub;            // the lane's first row; then every STEP rows
    constexpr int STEP = kTeam * RPL;
    long long place = 0;
    auto blocks = [&](int s) { return touched_blocks(p, s); };
    const int b = kMany ? find_item_cta(blockIdx.x, p.B, &place, blocks) : find_item(blockIdx.x, p.B, &place, blocks);
    if (b < 0) return;
    const int2 range = row_range(p.cu_new, b, p.n_new);
    const int past = p.past[b];
    const int i = past / BLOCK + static_cast<int>(place);                    // the sequence's block
    const int page = block_of(p.c.table, p.c.max_blocks, p.c.num_blocks, b, i);
    if (page < 0) return;
    // tokens [t0, t1) of the sequence are new and in this block
    const int t0 = max(past, i * BLOCK), t1 = min(past + (range.y - range.x), (i + 1) * BLOCK);
    const int o0 = t0 - i * BLOCK, n = t1 - t0;                 // offset of the first new row; rows
    // the block's heads, K's and then V's: neighbours, whose rows share lines, side by side
    [[maybe_unused]] int turn = 0;
    for (int job = blockIdx.y * (WARPS / kTeam) + team; job < 2 * p.c.H; job += gridDim.y * (WARPS / kTeam)) {
        const int kv = job >= p.c.H, head = job - kv * p.c.H;
        const __half *src = p.x[kv] + static_cast<size_t>(range.x + (t0 - past)) * p.ld[kv] + head * D + col;
        const size_t at = static_cast<size_t>(page) * p.c.H + head;
        int8_t *dst = p.c.codes[kv] + at * BLOCK * D;
        const float old = o0 > 0 ? p.c.scale[kv][at] : 0.0f;

        uint4 v[kHold];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int r = k * STEP + first;
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (r < n) v[k] = __ldg(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(r) * p.ld[kv]));
        }
#pragma unroll
        for (int k = 0; k < kHold; ++k) m = max_bits(v[k], m);
        for (int r = kHold * STEP + first; kHold * STEP < BLOCK && r < n; r += STEP)
            m = max_bits(__ldg(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(r) * p.ld[kv])), m);
        m = warp_max(max(m & 0xFFFFu, m >> 16));
        if constexpr (kTeam > 1) {
            __shared__ uint32_t tops[2][WARPS];      // in turn: a warp may be a job ahead
            if (lane == 0) tops[turn][team * kTeam + part] = m;
            static_assert(WARPS == 2 * kTeam, "two teams");
            if (team == 0)                             // (and all have read old)
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kTeam) : "memory");
            else
                asm volatile("bar.sync 2, %0;" ::"n"(32 * kTeam) : "memory");
#pragma unroll
            for (int k = 0; k < kTeam; ++k) m = max(m, tops[turn][team * kTeam + k]);
            turn ^= 1;
        }
        // non-negative floats order like their bits, and a NaN stays on top
        const uint32_t top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
        const bool grown = top > __float_as_uint(old);
        const float scale = grown ? __uint_as_float(top) : old;
        if (part == 0 && lane == 0) p.c.scale[kv][at] = scale;
        if (grown && old > 0.0f) {
            // the codes already there, four rows of D = 128 (eight of 64) a load
            const float ratio = __fdiv_rn(old, scale);
            for (int e = (part * 32 + lane) * 16; e < o0 * D; e += 512 * kTeam) {
                uint4 q = *reinterpret_cast<const uint4 *>(dst + e);
                uint32_t *w = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t out = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float c = static_cast<float>(static_cast<int8_t>((w[j] >> (8 * k)) & 0xFFu));
                        out |= (static_cast<uint32_t>(quant_code(c, ratio)) & 0xFFu) << (8 * k);
                    }
                    w[j] = out;
                }
                *reinterpret_cast<uint4 *>(dst + e) = q;
            }
        }
        const float inv = recip127(scale);
        dst += static_cast<size_t>(o0) * D + col;
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            const int r = k * STEP + first;
            if (r < n) *reinterpret_cast<uint2 *>(dst + r * D) = codes8(v[k], inv);
        }
        for (int r = kHold * STEP + first; kHold * STEP < BLOCK && r < n; r += STEP)
            *reinterpret_cast<uint2 *>(dst + r * D) =
                codes8(__ldg(reinterpret_cast<const uint4 *>(src + static_cast<size_t>(r) * p.ld[kv])), inv);
    }
}

struct GatherParams {
    Cache c;
    __half *out[2];                  // K, V: [rows, H, D]
    int rows, B;
    const int32_t *cu;               // [B+1]: sequence b's tokens are rows cu[b] .. cu[b+1]
};

// One warp per (block, head, K or V): fp16_rn(code * fl32(scale/127)).
template <int D, bool kMany>
__global__ void __launch_bounds__(32 * WARPS) kv_gather_kernel(const __grid_constant__ GatherParams p) {
    constexpr int LANES = D / 8;
    constexpr int RPL = 32 / LANES;
    constexpr int kAhead = 8;                      // loads in flight per lane
    const int lane = threadIdx.x & 31;
    const int sub = lane / LANES, col = (lane % LANES) * 8;
    const int job = blockIdx.y * WARPS + (threadIdx.x >> 5);
    long long place = 0;
    auto blocks = [&](int s) {
        const int2 r = row_range(p.cu, s, p.rows);
        return (r.y - r.x + BLOCK - 1) / BLOCK;
    };
    const int b = kMany ? find_item_cta(blockIdx.x, p.B, &place, blocks) : find_item(blockIdx.x, p.B, &place, blocks);
    if (b < 0 || job >= 2 * p.c.H) return;
    const int kv = job >= p.c.H, head = job - kv * p.c.H;        // neighbours share lines of their rows
    const int2 range = row_range(p.cu, b, p.rows);
    const int i = static_cast<int>(place);
    const int page = block_of(p.c.table, p.c.max_blocks, p.c.num_blocks, b, i);
    if (page < 0) return;
    const int n = min(BLOCK, range.y - range.x - i * BLOCK);
    const size_t at = static_cast<size_t>(page) * p.c.H + head;
    const int8_t *src = p.c.codes[kv] + at * BLOCK * D + col;
    __half *dst = p.out[kv] + (static_cast<size_t>(range.x + i * BLOCK) * p.c.H + head) * D + col;
    const float step = __fdiv_rn(p.c.scale[kv][at], 127.0f);
    for (int r0 = 0; r0 < n; r0 += kAhead * RPL) {
        uint2 q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * RPL + sub;
            q[k] = make_uint2(0u, 0u);
            if (r < n) q[k] = *reinterpret_cast<const uint2 *>(src + r * D);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k * RPL + sub;
            __half2 h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = (e < 2 ? q[k].x : q[k].y) >> (16 * (e & 1));
                h[e] = __floats2half2_rn(__fmul_rn(static_cast<float>(static_cast<int8_t>(w & 0xFFu)), step),
                                         __fmul_rn(static_cast<float>(static_cast<int8_t>((w >> 8) & 0xFFu)), step));
            }
            if (r < n)
                *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(r) * p.c.H * D) = *reinterpret_cast<uint4 *>(h);
        }
    }
}

}  // namespace kv
}  // namespace i8r

// Causal attention over packed prompts on the 5th-generation tensor cores.
//
// For query row i of a sequence with nq queries and nk keys (nk - nq of them
// from before the queries; row i sees keys 0 .. i + nk - nq):
//   x_ik = scale * Q_i . K_k,   O_i = sum_k e^(x_ik - m_i) V_k / sum_k e^(x_ik - m_i)
// in one pass over the keys with a running reference m_i and sum, so that the
// n x n scores never leave the SM.
//
// A CTA takes 256 query rows of one (sequence, head) as two tiles of 128.  Per
// 128 keys and tile:  S = Q K^T  (tcgen05.mma, fp32 in tensor memory, both
// operands K-major from TMA tiles);  four warps turn S into P = e^(x - m), one
// thread per row (a TMEM lane), fp16, written over S;  O += P V with P read from
// tensor memory and V as the MN-major operand straight from its row-major tile.
// The two tiles take turns: while one tile's warps do exponentials, the tensor
// cores do the other tile's two products.  Both tiles share each K and V tile.
//
// Per 128 keys and tile the products take 2 * 128 * 128 * D multiply-adds (1024
// cycles at D = 128) and the 128 * 128 exponentials 1024 cycles of the special
// function units: both pipes have to be kept busy, and neither can go below
// half of the time.  m_i is only raised (and O rescaled, by the softmax warps)
// when a row's maximum has grown by more than 2^8: e^(x-m) then stays below 256,
// which fp16 and the fp32 sums hold as exactly as values below 1.  P and its sum are
// 2^7 times that, below 2^15: a weight down to 2^-21 of the reference is a normal fp16
// number and is rounded by 2^-32 of it below that.  (With 1 at the reference, weights
// below 2^-25 were lost, 131072 of which are 0.4 % of the result.)
//
// What a mask leaves out must not be multiplied by zero: 0 * NaN is NaN.  Scores
// are replaced, not scaled, and on the one to three steps of a piece that a mask
// cuts, a warp looks for infinities and NaN among V's rows; where there is one, that
// step's P V is summed by the softmax warps over the visible keys alone.
//
// CTAs are persistent and everything crosses from one 256-row piece of work to the
// next: the next Q, K and V are loaded and its first scores computed while the last
// one's sums are scaled and stored.  Roles: warps 0-3 and 4-7 the two tiles' softmax,
// 8 the TMA producer, 9 and 10 the tiles' MMA issuers (a whole warp in step, so that
// operands stay in uniform registers; one warp for both tiles needed about 2000
// cycles for a tile's step of 1024), 11 finds the work and looks over V for what a
// mask must hide.  Every wait is bounded (timeout -> device status word).
//
// Measured: 8192 tokens, 40 query and 8 key heads of 128: 556 us, 1237 TFLOP/s (75 %
// of the dense 16-bit peak); 4 prompts of 1024, 96 heads: 167 to 172 us; 12 of 300: 160
// to 168 us; 200 tokens, 16 heads of 64: 12 to 14 us.  A step of both tiles takes about 3150 cycles
// (exponentials 1770 for a tile in its turn, then 1350 until its next scores are
// there), of 2048 that either pipe needs; a piece adds about 6000 to its steps.
#pragma once

#include "attention_decode.cuh"
#include "device_common.cuh"
#include "kv_cache.cuh"

namespace i8r {
namespace attn {

constexpr int PT = 128;                        // query rows per tile, keys per step
constexpr int PROMPT_ROWS = 2 * PT;            // query rows per CTA
constexpr int PROMPT_THREADS = 384;            // 8 softmax warps and four others
// Registers: 384 threads are launched with 168 each; the softmax warps take 216
// (a row's 128 scores stay in them) and the other four 72.
constexpr int PROMPT_LAUNCH_REGS = 168, SOFTMAX_REGS = 216, OTHER_REGS = 72;
static_assert(SOFTMAX_REGS * 256 + OTHER_REGS * 128 <= PROMPT_LAUNCH_REGS * PROMPT_THREADS, "more registers than launched with");
constexpr uint32_t PROMPT_TMEM = 512;
constexpr float PROMPT_RAISED = 7.0f;          // log2 of a weight at its row's reference
constexpr float RAISE = 8.0f;                  // log2 of how far a row may exceed its reference

constexpr int OUT_BYTES = 32 * 128;            // a softmax warp's rows on their way out, 64 columns at a time

template <int D>
struct PromptShape {
    static constexpr int CHUNKS = D / 64;                      // 128-byte swizzle spans of a row
    static constexpr int CHUNK_BYTES = PT * 128;
    static constexpr int TILE_BYTES = CHUNKS * CHUNK_BYTES;    // a Q, K or V tile
    static constexpr int STAGES = D == 128 ? 4 : 10;
    static constexpr size_t SMEM = 1024 + (2 + STAGES) * TILE_BYTES + 8 * OUT_BYTES + 1024;
};

struct PromptParams {
    __half *O;
    long long ldo;
    int N, M, B, Hq, H, G;                     // query rows, key rows, sequences, heads, group
    const int32_t *cu_q, *cu_k;
    float scale_log2;                          // |scale| * log2(e), not 0
    uint32_t negate;                           // idesc bit: scale < 0
};

// 256 query rows of one (sequence, head).
struct PromptWork {
    int row, rows;                             // first row of Q and O; rows of the sequence from there on
    int key, head;                             // first row of K and V
    int seen;                                  // the last of the sequence's keys that the first row sees (may be < 0)
    int steps[2];                              // steps of 128 keys for each tile; -1: no more work
};
// The first step that the mask cuts for a tile whose first row sees keys up to `seen`;
// from the first tile's on there are at most kCuts steps.
constexpr int kCuts = 3;
__device__ __forceinline__ int first_cut(int seen) { return seen + 1 > 0 ? (seen + 1) / PT : 0; }

constexpr int kEarly = 6;                      // of a step's eight MMAs over 16 keys of P, those that need not wait for the last
constexpr int kWorkSlots = 4;                  // pieces of work known at a time
// Barriers that complete once per piece of work have parity (work & 1); those of a
// work slot (work / kWorkSlots) & 1.
struct PromptBarriers {
    uint64_t full[10], empty[10];              // the K/V ring
    uint64_t q_full[2], q_empty[2];            // a tile's queries
    uint64_t s_full[2], p_ready[2][2];         // scores; P of the first kEarly * 16 keys, of the others (once per step)
    uint64_t o_full[2], o_empty[2];            // the sums
    uint64_t turn[2][4];                       // tile i's warp has done its exponentials: the other tile's may begin
    uint64_t asked[kWorkSlots][kCuts], scan[kWorkSlots][kCuts];      // V of a cut step: asked for, looked over
    uint64_t work_full[kWorkSlots], work_empty[kWorkSlots];
    uint64_t drain[2];
    PromptWork work[kWorkSlots];
    uint32_t tmem_base;
    int abort;
    int dirty[kWorkSlots][kCuts], skip[2];     // a cut step's V is not finite; the step (counted through) whose P V is done
};
static_assert(sizeof(PromptBarriers) <= 1024, "barrier block outgrew its shared-memory reserve");

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

// The MMAs with descriptors given as their low halves (address and leading
// dimension; the high half is the same for every operand here): one addition an
// operand.  Called by a whole warp; one lane issues.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);    // 8 rows 1024 B apart, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t address, uint32_t lbo) { return (address >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
        "r"(accumulate), "r"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a_tmem), "r"(b), "r"(idesc),
        "r"(accumulate), "r"(kDescHigh)
        : "memory");
}

__device__ __forceinline__ void commit_elected(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// A wait of a whole warp.  All lanes look, about 40 cycles a look (a try_wait sleeps
// until the barrier's phase ends or some time has passed); lane 0's look and its
// broadcast, which the bounded wait is made of, take 240.
__device__ __forceinline__ bool ready(uint64_t *bar, uint32_t parity, volatile int *abort, int code) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    return warp_wait(bar, parity, abort, code);
}

// First row, within work n, of tile i's 128: the tiles change places from one piece of work
// to the next.  The second 128 rows see one step more than the first, and a short piece has
// no second 128: so the tile that had less of a piece has more of the next, and is already
// at it while the other one finishes.
__device__ __forceinline__ int place_of(int i, int n) { return (i ^ (n & 1)) * PT; }

__device__ __forceinline__ __half2 largest(__half2 m, uint32_t x) {
    return __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2 *>(&x)));
}

// P V of one step over the keys that each row sees, without the tensor cores: O (in
// tensor memory at t_o; zeros before the first step) += sum over keys 0 .. seen of
// this lane's P (at t_s) and V's rows (128-byte-swizzled 64-column chunks).  For the
// rare step whose V holds infinities or NaN that some rows do not see.
template <int D>
__device__ __forceinline__ void values_seen(uint32_t t_s, uint32_t t_o, const uint8_t *v, bool accumulate, int seen) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
        if (accumulate) {
            tmem_ld32(t_o + 32 * c, o);
            tmem_wait_ld();
        }
#pragma unroll 1
        for (int k = 0; k < PT; ++k) {
            uint32_t pp;
            tmem_ld1(t_s + k / 2, pp);
            tmem_wait_ld();
            const float2 pf = __half22float2(*reinterpret_cast<const __half2 *>(&pp));
            if (k <= seen) {
                const float pk = (k & 1) ? pf.y : pf.x;
                const uint8_t *src = v + (c >> 1) * PromptShape<D>::CHUNK_BYTES + k * 128;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(src + (((4 * (c & 1) + u) ^ (k & 7)) << 4));
                    const __half2 *hv = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = __half22float2(hv[e]);
                        uint32_t &o0 = o[8 * u + 2 * e], &o1 = o[8 * u + 2 * e + 1];
                        o0 = __float_as_uint(fmaf(pk, f.x, __uint_as_float(o0)));
                        o1 = __float_as_uint(fmaf(pk, f.y, __uint_as_float(o1)));
                    }
                }
            }
            __syncwarp();
        }
        tmem_st32(t_o + 32 * c, o);
    }
    tmem_wait_st();
}

template <int D>
__global__ void __launch_bounds__(PROMPT_THREADS, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptParams p) {
    using Shape = PromptShape<D>;
    constexpr int STAGES = Shape::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + 2 * Shape::TILE_BYTES;
    uint8_t *out = ring + STAGES * Shape::TILE_BYTES;
    PromptBarriers *bars = reinterpret_cast<PromptBarriers *>(out + 8 * OUT_BYTES);
    volatile int *abort = &bars->abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 2);                     // both tiles' MMAs
        }
        for (int s = 0; s < kWorkSlots; ++s) {
            for (int c = 0; c < kCuts; ++c) {
                mbar_init(&bars->asked[s][c], 1);
                mbar_init(&bars->scan[s][c], 1);
            }
            mbar_init(&bars->work_full[s], 1);
            mbar_init(&bars->work_empty[s], 11);               // 8 softmax warps, producer, 2 MMA issuers
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 1);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_ready[i][0], 4);
            mbar_init(&bars->p_ready[i][1], 4);
            mbar_init(&bars->o_full[i], 1);
            mbar_init(&bars->o_empty[i], 4);
            for (int k = 0; k < 4; ++k) mbar_init(&bars->turn[i][k], 1);
            bars->skip[i] = -1;
        }
        mbar_init(&bars->drain[0], 1);
        mbar_init(&bars->drain[1], 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_v);
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, PROMPT_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bars->tmem_base, 0);

    // the next piece of work, for every lane of a warp; false when there is none or the CTA gives up
    auto take = [&](int n, PromptWork *w) {
        if (!ready(&bars->work_full[n % kWorkSlots], (n / kWorkSlots) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT)) return false;
        *w = bars->work[n % kWorkSlots];
        return w->steps[0] >= 0;
    };
    auto give_back = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->work_empty[n % kWorkSlots]);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == 11) {
            // -------------------------------------------------------- the work, this CTA's share of it.
            // In order of their length (in 256 keys: the level), the longest pieces first, dealt to
            // the CTAs there and back; neighbours are the heads of one tile, which share keys and
            // values.  Sequence s has its tile t at level t + before(s), for each of its tiles.
            // Levels that no sequence has a tile at are passed over: a look at all sequences costs
            // about 0.4 us for each 32 of them (one row on 2^20 keys beside 4000 short prompts: 203 ms
            // with a look at every level down to theirs, 11 with this, which is the long row alone).
            auto span = [&](int s) {                         // its levels [x, y)
                const int2 q = kv::row_range(p.cu_q, s, p.N), k = kv::row_range(p.cu_k, s, p.M);
                const int nq = q.y - q.x, before = max(0, k.y - k.x - nq) / PROMPT_ROWS;
                return make_int2(before, before + (nq + PROMPT_ROWS - 1) / PROMPT_ROWS);
            };
            int level = 0, below = -1;                       // this level; the next one with a tile, -1: none
            long long base = 0, here = 0;                    // pieces (without heads) of the levels above, of this one
            int2 mine = make_int2(0, 0);                     // this lane's sequence, when a warp holds them all
            int from = 0;                                    // else how far the search on this level has come
            long long passed = 0;
            for (int s = lane; s < p.B; s += 32) {
                mine = span(s);
                if (mine.y > mine.x) below = max(below, mine.y - 1);
            }
            const bool few = p.B <= 32;
            below = __reduce_max_sync(0xFFFFFFFFu, below);   // the highest (no piece before it: here is 0)
            auto publish = [&](int n) {                      // false: there is no more, or the CTA gives up
                const int turn = (n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
                const long long item = turn + static_cast<long long>(n) * gridDim.x;
                const long long piece = item >> 31 ? item / p.Hq : static_cast<uint32_t>(item) / static_cast<uint32_t>(p.Hq);
                while (level >= 0 && piece >= base + here) {
                    base += here;
                    level = below;
                    if (level < 0) break;
                    int count = 0, next = -1;
                    auto look = [&](const int2 &v) {
                        count += level >= v.x && level < v.y;
                        if (v.x < min(v.y, level)) next = max(next, min(v.y, level) - 1);
                    };
                    if (few) look(mine);
                    for (int s = lane; s < p.B && !few; s += 32) look(span(s));
                    here = __reduce_add_sync(0xFFFFFFFFu, count);
                    below = __reduce_max_sync(0xFFFFFFFFu, next);
                    from = 0;
                    passed = 0;
                }
                PromptWork w{};
                w.steps[0] = -1;
                if (level >= 0) {
                    int b;
                    if (few) {                               // the (piece - base)-th sequence that has a tile here
                        const bool here_too = level >= mine.x && level < mine.y;
                        const unsigned set = __ballot_sync(0xFFFFFFFFu, here_too);
                        const int rank = __popc(set & ((1u << lane) - 1u));
                        b = __ffs(__ballot_sync(0xFFFFFFFFu, here_too && rank == static_cast<int>(piece - base))) - 1;
                    } else {
                        long long place = 0;
                        b = kv::find_item(piece - base, p.B, &place, [&](int s) {
                            const int2 v = span(s);
                            return level >= v.x && level < v.y ? 1 : 0;
                        }, &from, &passed);
                    }
                    const int2 qr = kv::row_range(p.cu_q, b, p.N), kr = kv::row_range(p.cu_k, b, p.M);
                    const int nq = qr.y - qr.x, off = kr.y - kr.x - nq;
                    const int first = (level - max(0, off) / PROMPT_ROWS) * PROMPT_ROWS;
                    w.row = qr.x + first;
                    w.rows = nq - first;
                    w.key = kr.x;
                    w.head = static_cast<int>(item - piece * p.Hq);
                    w.seen = first + off;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // what the tile's last row sees
                        const int at = place_of(i, n), keys = at < w.rows ? min(at + PT, w.rows) + w.seen : 0;
                        w.steps[i] = keys > 0 ? (keys + PT - 1) / PT : 0;
                    }
                }
                const int slot = n % kWorkSlots;
                if (n >= kWorkSlots &&
                    !ready(&bars->work_empty[slot], (n / kWorkSlots - 1) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT))
                    return false;
                if (lane == 0) {
                    bars->work[slot] = w;
                    mbar_arrive(&bars->work_full[slot]);
                }
                __syncwarp();
                return level >= 0;
            };
            int tile = 0, given = 0;                         // tiles of the ring so far; pieces told
            bool more = true, ok = true;
            auto tell = [&] {
                if (more && (more = publish(given))) ++given;
            };
            tell();
            tell();                                          // a search hides behind the piece before it
            for (int n = 0; ok && n < given; ++n) {
                // infinities and NaN in V of the steps that a mask cuts
                const int slot = n % kWorkSlots, parity = (n / kWorkSlots) & 1;
                const PromptWork w = bars->work[slot];
                const int all = max(w.steps[0], w.steps[1]), cut = first_cut(w.seen);
                for (int c = 0; ok && c < kCuts; ++c) {
                    // This warp does not follow the ring's turns, and a parity cannot tell a
                    // turn from the one two before: once the producer has asked for this one,
                    // it is the one that full[] completes next.
                    ok = ready(&bars->asked[slot][c], parity, abort, I8R_DEV_PIPELINE_TIMEOUT);
                    // largest magnitudes; a NaN stays
                    __half2 top[4] = {};
                    if (ok && cut + c < all) {
                        const int k = tile + 2 * (cut + c) + 1;
                        ok = ready(&bars->full[k % STAGES], (k / STAGES) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT);
                        const uint4 *v = reinterpret_cast<const uint4 *>(ring + k % STAGES * Shape::TILE_BYTES) + lane;
#pragma unroll 4
                        for (int e = 0; e < Shape::TILE_BYTES / 512; e += 4)
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const uint4 x = v[(e + z) * 32];
                                top[0] = largest(top[0], x.x);
                                top[1] = largest(top[1], x.y);
                                top[2] = largest(top[2], x.z);
                                top[3] = largest(top[3], x.w);
                            }
                    }
                    const __half2 all4 = __hmax2_nan(__hmax2_nan(top[0], top[1]), __hmax2_nan(top[2], top[3]));
                    const uint32_t m = *reinterpret_cast<const uint32_t *>(&all4);
                    const bool bad = __any_sync(0xFFFFFFFFu, (m >> 16 & 0x7FFFu) >= 0x7C00u || (m & 0x7FFFu) >= 0x7C00u);
                    if (lane == 0) {
                        bars->dirty[slot][c] = bad;
                        mbar_arrive(&bars->scan[slot][c]);
                    }
                }
                tile += 2 * all;
                tell();
            }
        } else if (warp == 8) {
            // -------------------------------------------------------- producer
            int tile = 0;
            bool ok = true;
            int q_loaded[2] = {-1, -1};                      // the last work whose queries were asked for
            PromptWork w;
            int n = 0;
            for (; ok && take(n, &w); ++n) {
                const int all = max(w.steps[0], w.steps[1]), x = (w.head / p.G) * D, cut = first_cut(w.seen);
                auto load_kv = [&](int k) {                  // K_0, V_0, K_1, V_1, ...
                    const int s = (tile + k) % STAGES, turn = (tile + k) / STAGES;
                    ok = ok && (turn == 0 || ready(&bars->empty[s], (turn - 1) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT));
                    if (!ok) return;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars->full[s], Shape::TILE_BYTES);
                        for (int c = 0; c < Shape::CHUNKS; ++c)
                            tma_load_2d(ring + s * Shape::TILE_BYTES + c * Shape::CHUNK_BYTES, (k & 1) ? &map_v : &map_k,
                                        &bars->full[s], x + 64 * c, w.key + (k >> 1) * PT);
                        if ((k & 1) && (k >> 1) >= cut) mbar_arrive(&bars->asked[n % kWorkSlots][(k >> 1) - cut]);
                    }
                    __syncwarp();
                };
                // K_0, Q, V_0: what the first scores need is free before V_0's place is
                int k = 0;
                for (; ok && k < 1 && k < 2 * all; ++k) load_kv(k);
                for (int i = 0; ok && i < 2; ++i) {
                    ok = n == 0 || ready(&bars->q_empty[i], (n - 1) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars->q_full[i], w.steps[i] > 0 ? Shape::TILE_BYTES : 0);
                        for (int c = 0; w.steps[i] > 0 && c < Shape::CHUNKS; ++c)
                            tma_load_2d(smem + i * Shape::TILE_BYTES + c * Shape::CHUNK_BYTES, &map_q, &bars->q_full[i],
                                        w.head * D + 64 * c, w.row + place_of(i, n));
                    }
                    q_loaded[i] = n;
                    __syncwarp();
                }
                for (; ok && k < 2 * all; ++k) load_kv(k);
                tile += k;                                   // (what was asked for, when giving up)
                if (ok && lane == 0)
                    for (int c = max(0, all - cut); c < kCuts; ++c) mbar_arrive(&bars->asked[n % kWorkSlots][c]);      // no such step
                if (ok) give_back(n);
            }
            if (*abort && lane == 0) {
                // given up: let the loads in flight land before the CTA leaves
                volatile int never = 0;
                for (int i = 0; i < 2; ++i)
                    if (q_loaded[i] >= 0) mbar_wait(&bars->q_full[i], q_loaded[i] & 1, &never, 0);
                for (int k = max(0, tile - STAGES); k < tile; ++k)
                    mbar_wait(&bars->full[k % STAGES], (k / STAGES) & 1, &never, 0);
            }
        } else {
            // -------------------------------------------------------- MMA issuer
            const uint32_t id_s = idesc_f16(PT, PT, false, false) | p.negate;
            const uint32_t id_o = idesc_f16(PT, D, false, true);
            const int i = warp - 9;                          // the tile
            const uint32_t q_base = desc_low(smem_u32(smem + i * Shape::TILE_BYTES), 16), ring_base = smem_u32(ring);
            const uint32_t t_s = tmem + i * PT, t_o = tmem + 2 * PT + i * D;
            int tile = 0, done = 0;                          // tiles of the ring, steps of this tile before this work
            bool ok = true;
            auto landed = [&](int k) {                       // each of the ring's tiles, in order
                return ready(&bars->full[(tile + k) % STAGES], ((tile + k) / STAGES) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT);
            };
            auto scores = [&](int j) {
                const uint32_t k = desc_low(ring_base + (tile + 2 * j) % STAGES * Shape::TILE_BYTES, 16);
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = ((kk >> 2) * Shape::CHUNK_BYTES + (kk & 3) * 32) >> 4;
                    mma_ss(t_s, q_base + o, k + o, id_s, kk != 0);
                }
                commit_elected(&bars->s_full[i]);
            };
            PromptWork w;
            for (int n = 0; ok && take(n, &w); ++n) {
                const int steps = __shfl_sync(0xFFFFFFFFu, w.steps[i], 0), all = max(w.steps[0], w.steps[1]);
                const int cut = first_cut(w.seen);
                give_back(n);
                ok = ready(&bars->q_full[i], n & 1, abort, I8R_DEV_PIPELINE_TIMEOUT);
                if (ok && steps > 0) {
                    ok = landed(0);
                    if (ok) scores(0);
                }
                if (ok && steps <= 1) commit_elected(&bars->q_empty[i]);
                // the sums are free once the work before has been read out of them
                ok = ok && (n == 0 || ready(&bars->o_empty[i], (n - 1) & 1, abort, I8R_DEV_TMEM_TIMEOUT));
                if (ok && steps == 0) commit_elected(&bars->o_full[i]);          // a tile without keys
                for (int j = 0; ok && j < all; ++j) {
                    // Both issuers pass every tile of the ring, also those that their own tile has no step
                    // for (waiting for its turn: a commit must not count for the turn before).
                    if (j >= steps) {
                        for (int k = 2 * j; ok && k < 2 * j + 2; ++k)
                            if ((ok = landed(k))) commit_elected(&bars->empty[(tile + k) % STAGES]);
                        continue;
                    }
                    commit_elected(&bars->empty[(tile + 2 * j) % STAGES]);       // K_j: its scores are issued
                    const bool more = j + 1 < steps;
                    const uint32_t v = desc_low(ring_base + (tile + 2 * j + 1) % STAGES * Shape::TILE_BYTES, Shape::CHUNK_BYTES);
                    // three quarters of P while the softmax warps are at the last one
                    ok = landed(2 * j + 1) && (!more || landed(2 * j + 2));
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        ok = ok && ready(&bars->p_ready[i][part], (done + j) & 1, abort, I8R_DEV_TMEM_TIMEOUT);
                        if (!ok || (j >= cut && *static_cast<volatile int *>(&bars->skip[i]) == done + j)) continue;
                        tc_fence_after_sync();
#pragma unroll
                        for (int kk = part ? kEarly : 0; kk < (part ? PT / 16 : kEarly); ++kk)
                            mma_ts(t_o, t_s + kk * 8, v + (kk * 16 * 128 >> 4), id_o, (j | kk) != 0);
                    }
                    if (!ok) break;
                    if (more) {
                        scores(j + 1);
                        if (j + 2 == steps) commit_elected(&bars->q_empty[i]);   // its last scores
                    } else {
                        commit_elected(&bars->o_full[i]);
                    }
                    commit_elected(&bars->empty[(tile + 2 * j + 1) % STAGES]);
                }
                tile += 2 * all;
                done += steps;
            }
            volatile int never = 0;
            commit_elected(&bars->drain[i]);
            if (lane == 0) mbar_wait(&bars->drain[i], 0, &never, 0);
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax, one row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
        const int i = warp >> 2, quad = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lanes + i * PT, t_o = tmem + lanes + 2 * PT + i * D;
        const float sl2 = p.scale_log2;
        int tile = 0, done = 0;                                 // tiles of the ring, steps of this tile before this work
        int turns = 0;                                          // steps of both tiles before this work
        bool ok = true;
        PromptWork w;
        for (int n = 0; ok && take(n, &w); ++n) {
            const int steps = w.steps[i], cut0 = first_cut(w.seen), cut = first_cut(w.seen + place_of(i, n));
            const int lim = w.seen + place_of(i, n) + quad * 32 + lane;     // the last key the row sees
            const int both = min(w.steps[0], w.steps[1]);
            // p = 2^(x * sl2 + ref): ref is PROMPT_RAISED - reference (log2 units), infinite before the first
            // key.  Whether a row has outgrown it is asked of the largest p's own exponent, rounded as
            // it will be, so that no p exceeds 2^(PROMPT_RAISED + RAISE) however large the scores are.
            float ref = INFINITY, l = 0.0f;
            for (int j = 0; j < steps; ++j) {
                ok = ready(&bars->s_full[i], (done + j) & 1, abort, I8R_DEV_TMEM_TIMEOUT);
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, r[c]);
                tmem_wait_ld();
                // a step that every row of the tile sees whole needs no mask
                if (j >= cut) {
                    const int seen = lim - j * PT;              // columns 0 .. seen stay
#pragma unroll
                    for (int e = 0; e < PT; ++e)
                        if (e > seen) r[e >> 5][e & 31] = 0xFF800000u;  // -infinity
                }
                auto x = [&](int e) { return __uint_as_float(r[e >> 5][e & 31]); };
                float top[4] = {x(0), x(1), x(2), x(3)};
#pragma unroll
                for (int e = 4; e < PT - 4; e += 8)
#pragma unroll
                    for (int c = 0; c < 4; ++c) top[c] = max3(top[c], x(e + 2 * c), x(e + 2 * c + 1));
                const float mx = fmaxf(max3(max3(top[0], top[1], x(PT - 4)), max3(top[2], top[3], x(PT - 3)), x(PT - 2)), x(PT - 1));
                const float most = fmaf(mx, sl2, ref);          // (NaN where nothing was seen, now or before)
                if (__any_sync(0xFFFFFFFFu, most > PROMPT_RAISED + RAISE)) {
                    const float to = most > PROMPT_RAISED ? fmaf(-mx, sl2, PROMPT_RAISED) : ref;
                    const float alpha = most > PROMPT_RAISED ? ex2(to - ref) : 1.0f;
                    l *= alpha;
                    ref = to;
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(t_o + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(t_o + 32 * c, o);
                        }
                    }
                }
                // The two tiles take turns at the exponentials (their warps share the special
                // function units, and would fall in step: both at the exponentials, then both
                // waiting for the tensor cores); the one with the second 128 rows, which was done
                // first with the work before, leads.  Nothing depends on it but time.
                const int before = j - ((i ^ n) & 1);
                if (before >= 0 && before < both)
                    ok = ready(&bars->turn[1 - i][quad], (turns + before) & 1, abort, I8R_DEV_TMEM_TIMEOUT);
                if (!ok) break;
                // (a row that has seen nothing yet has all -inf)
                const float add = ref == INFINITY ? 0.0f : ref;
                const uint64_t sl22 = pack2(sl2, sl2), ref2 = pack2(add, add);
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t out[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (c == 3 && e == 6) {                 // by now the first three quarters are stored
                            tmem_wait_st();
                            tc_fence_before_sync();
                            __syncwarp();
                            if (j < cut && lane == 0) mbar_arrive(&bars->p_ready[i][0]);
                        }
                        // the other tile's turn: told ahead of the end, for the time that the telling takes
                        if (c == 3 && e == 6 && j < both && lane == 0) mbar_arrive(&bars->turn[i][quad]);
                        const float2 y = unpack2(fma2(pack2(x(32 * c + 2 * e), x(32 * c + 2 * e + 1)), sl22, ref2));
                        const float p0 = ex2(y.x), p1 = ex2(y.y);
                        sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                        const __half2 h2 = __floats2half2_rn(p0, p1);
                        out[e] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    tmem_st16(t_s + 16 * c, out);
                }
                const float2 s2 = unpack2(add2(sum[0], sum[1]));
                l += s2.x + s2.y;
                tmem_wait_st();
                bool dirty = false;
                if (j >= cut) {                                 // what V holds is known by now, or soon
                    ok = ready(&bars->scan[n % kWorkSlots][j - cut0], (n / kWorkSlots) & 1, abort, I8R_DEV_TMEM_TIMEOUT);
                    if (!ok) break;
                    dirty = *static_cast<volatile int *>(&bars->dirty[n % kWorkSlots][j - cut0]) != 0;
                    if (dirty && lane == 0) *static_cast<volatile int *>(&bars->skip[i]) = done + j;
                }
                if (dirty)
                    values_seen<D>(t_s, t_o, ring + (tile + 2 * j + 1) % STAGES * Shape::TILE_BYTES, j > 0, lim - j * PT);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (j >= cut) mbar_arrive(&bars->p_ready[i][0]);
                    mbar_arrive(&bars->p_ready[i][1]);
                }
            }
            ok = ok && ready(&bars->o_full[i], n & 1, abort, I8R_DEV_TMEM_TIMEOUT);
            if (!ok) break;
            tc_fence_after_sync();
            // O / l in fp16, 64 columns at a time through shared memory (piece e, 16 bytes, of
            // row r in place e ^ (r % 8)), so that whole lines are written.  A row that sees no
            // key is zeros, whatever its tile's steps left.
            // A warp that has no row of the sequence only says that it has looked.
            const bool none = steps == 0 || lim < 0;            // (then what tensor memory holds is not looked at)
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint8_t *mine = out + warp * OUT_BYTES;
            // (read again: the loop above has no register to spare)
            const volatile PromptWork *again = &bars->work[n % kWorkSlots];
            const int rows = again->rows, row0 = place_of(i, n) + quad * 32;
            __half *dst = p.O + static_cast<size_t>(again->row + row0 + (lane >> 3)) * p.ldo + static_cast<size_t>(again->head) * D +
                          8 * (lane & 7);
            if (row0 >= rows) {
                tc_fence_before_sync();
                if (lane == 0) mbar_arrive(&bars->o_empty[i]);
            }
#pragma unroll
            for (int h = 0; h < D / 64 && row0 < rows; ++h) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    uint32_t o[32];
                    tmem_ld32(t_o + 64 * h + 32 * z, o);
                    tmem_wait_ld();
                    if (z == 1 && h + 1 == D / 64) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->o_empty[i]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 v;
                        uint32_t *f = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __half2 h2 = __floats2half2_rn(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                                                 __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                            f[k] = *reinterpret_cast<const uint32_t *>(&h2);
                        }
                        if (none) v = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(mine + lane * 128 + (((4 * z + e) ^ (lane & 7)) << 4)) = v;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = 4 * k + (lane >> 3);
                    const uint4 v = *reinterpret_cast<const uint4 *>(mine + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                    if (row0 + row < rows)
                        *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(4 * k) * p.ldo + 64 * h) = v;
                }
                __syncwarp();
            }
            tile += 2 * max(again->steps[0], again->steps[1]);
            turns += min(again->steps[0], again->steps[1]);
            done += steps;
            give_back(n);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, PROMPT_TMEM);
    }
}

}  // namespace attn
}  // namespace i8r

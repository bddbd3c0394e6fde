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
// which fp16 and the fp32 sums hold as exactly as values below 1.
//
// What a mask leaves out must not be multiplied by zero: 0 * NaN is NaN.  Scores
// are replaced, not scaled, and on the one or two steps of a tile that a mask
// cuts, the tile's warps look for infinities and NaN among V's rows; where there
// is one, that step's P V is summed by the warps over the visible keys alone.
//
// Roles: warps 0-3 and 4-7 the tiles' softmax, warp 8 the TMA producer, warp 9
// the MMA issuer.  Every wait is bounded (timeout -> device status word).
#pragma once

#include "attention_decode.cuh"
#include "device_common.cuh"
#include "kv_cache.cuh"

namespace i8r {
namespace attn {

constexpr int PT = 128;                        // query rows per tile, keys per step
constexpr int PROMPT_ROWS = 2 * PT;            // query rows per CTA
constexpr int PROMPT_THREADS = 320;
constexpr uint32_t PROMPT_TMEM = 512;
constexpr float RAISE = 8.0f;                  // log2 of how far a row may exceed its reference

template <int D>
struct PromptShape {
    static constexpr int CHUNKS = D / 64;                      // 128-byte swizzle spans of a row
    static constexpr int CHUNK_BYTES = PT * 128;
    static constexpr int TILE_BYTES = CHUNKS * CHUNK_BYTES;    // a Q, K or V tile
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr size_t SMEM = 1024 + (2 + STAGES) * TILE_BYTES + 512;
};

struct PromptParams {
    __half *O;
    long long ldo;
    int N, M, B, Hq, H, G;                     // query rows, key rows, sequences, heads, group
    const int32_t *cu_q, *cu_k;
    float scale_log2;                          // |scale| * log2(e), not 0
    uint32_t negate;                           // idesc bit: scale < 0
};

struct PromptBarriers {
    uint64_t full[10], empty[10];              // the K/V ring
    uint64_t q_full;
    uint64_t s_full[2], p_ready[2], o_full[2], scan[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int dirty_step[2], skip_step[2];
};
static_assert(sizeof(PromptBarriers) <= 512, "barrier block outgrew its shared-memory reserve");

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

// Whether any of eight fp16 values is an infinity or NaN (exponent all ones).
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (w[i] & 0x7C007C00u) >= 0x7C000000u || (w[i] & 0x00007C00u) == 0x00007C00u;
    return bad;
}

template <int D>
__global__ void __launch_bounds__(PROMPT_THREADS, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptParams p) {
    using Shape = PromptShape<D>;
    constexpr int STAGES = Shape::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // The longest tiles of a sequence first; neighbouring CTAs are the heads of one
    // tile, which share keys and values.
    const int head = blockIdx.x % p.Hq;
    long long place = 0;
    auto tiles = [&](int s) {
        const int2 r = kv::row_range(p.cu_q, s, p.N);
        return (r.y - r.x + PROMPT_ROWS - 1) / PROMPT_ROWS;
    };
    const int b = kv::find_item(blockIdx.x / p.Hq, p.B, &place, tiles);
    if (b < 0) return;
    const int2 qr = kv::row_range(p.cu_q, b, p.N), kr = kv::row_range(p.cu_k, b, p.M);
    const int nq = qr.y - qr.x, nk = kr.y - kr.x, off = nk - nq;
    const int first_row = (tiles(b) - 1 - static_cast<int>(place)) * PROMPT_ROWS;
    // steps of 128 keys: what the tile's last row sees
    int steps[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row0 = first_row + i * PT;
        const int seen = row0 < nq ? min(row0 + PT, nq) + off : 0;
        steps[i] = seen > 0 ? (seen + PT - 1) / PT : 0;
    }
    const int all = max(steps[0], steps[1]);

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + 2 * Shape::TILE_BYTES;
    PromptBarriers *bars = reinterpret_cast<PromptBarriers *>(ring + STAGES * Shape::TILE_BYTES);
    volatile int *abort = &bars->abort;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        mbar_init(&bars->q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_ready[i], 4);
            mbar_init(&bars->o_full[i], 1);
            mbar_init(&bars->scan[i], 4);
            bars->dirty_step[i] = bars->skip_step[i] = -1;
        }
        mbar_init(&bars->drain, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bars->tmem_base, PROMPT_TMEM);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && all > 0) {
            const int nt = steps[1] > 0 ? 2 : 1;
            mbar_arrive_expect_tx(&bars->q_full, nt * Shape::TILE_BYTES);
            for (int i = 0; i < nt; ++i)
                for (int c = 0; c < Shape::CHUNKS; ++c)
                    tma_load_2d(smem + i * Shape::TILE_BYTES + c * Shape::CHUNK_BYTES, &map_q, &bars->q_full,
                                head * D + 64 * c, qr.x + first_row + i * PT);
            const int x = (head / p.G) * D;
            int issued = 0;
            for (; issued < 2 * all; ++issued) {             // K_0, V_0, K_1, V_1, ...
                const int s = issued % STAGES;
                if (issued >= STAGES && !mbar_wait(&bars->empty[s], (issued / STAGES - 1) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT))
                    break;
                mbar_arrive_expect_tx(&bars->full[s], Shape::TILE_BYTES);
                for (int c = 0; c < Shape::CHUNKS; ++c)
                    tma_load_2d(ring + s * Shape::TILE_BYTES + c * Shape::CHUNK_BYTES, (issued & 1) ? &map_v : &map_k,
                                &bars->full[s], x + 64 * c, kr.x + (issued >> 1) * PT);
            }
            if (issued < 2 * all) {
                // given up: let the loads in flight land before the CTA leaves
                volatile int never = 0;
                mbar_wait(&bars->q_full, 0, &never, 0);
                for (int k = max(0, issued - STAGES); k < issued; ++k)
                    mbar_wait(&bars->full[k % STAGES], (k / STAGES) & 1, &never, 0);
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && all > 0) {
            const uint32_t id_s = idesc_f16(PT, PT, false, false) | p.negate;
            const uint32_t id_o = idesc_f16(PT, D, false, true);
            int got = -1;                                    // last ring tile known to have landed
            auto landed = [&](int k) {
                for (; got < k; ++got)
                    if (!mbar_wait(&bars->full[(got + 1) % STAGES], ((got + 1) / STAGES) & 1, abort,
                                   I8R_DEV_PIPELINE_TIMEOUT))
                        return false;
                tc_fence_after_sync();
                return true;
            };
            auto scores = [&](int i, int j) {
                const uint32_t a = smem_u32(smem + i * Shape::TILE_BYTES);
                const uint32_t k = smem_u32(ring + (2 * j) % STAGES * Shape::TILE_BYTES);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * Shape::CHUNK_BYTES + (kk & 3) * 32;
                    mma_f16(tmem + i * PT, smem_desc_sw128(a + o, 16, 1024), smem_desc_sw128(k + o, 16, 1024), id_s, kk != 0);
                }
                mma_commit(&bars->s_full[i]);
            };
            bool ok = mbar_wait(&bars->q_full, 0, abort, I8R_DEV_PIPELINE_TIMEOUT) && landed(0);
            if (ok) {
                for (int i = 0; i < 2; ++i)
                    if (steps[i] > 0) scores(i, 0);
                mma_commit(&bars->empty[0]);
            }
            for (int j = 0; ok && j < all; ++j) {
                for (int i = 0; ok && i < 2; ++i) {
                    if (j >= steps[i]) continue;
                    ok = mbar_wait(&bars->p_ready[i], j & 1, abort, I8R_DEV_TMEM_TIMEOUT) && landed(2 * j + 1);
                    if (!ok) break;
                    if (*static_cast<volatile int *>(&bars->skip_step[i]) != j) {
                        const uint32_t v = smem_u32(ring + (2 * j + 1) % STAGES * Shape::TILE_BYTES);
#pragma unroll
                        for (int kk = 0; kk < PT / 16; ++kk)
                            mma_f16_tmem_a(tmem + 2 * PT + i * D, tmem + i * PT + kk * 8,
                                           smem_desc_sw128(v + kk * 16 * 128, Shape::CHUNK_BYTES, 1024), id_o,
                                           (j | kk) != 0);
                    }
                    if (j + 1 == steps[i]) {
                        mma_commit(&bars->o_full[i]);
                    } else {
                        ok = landed(2 * j + 2);
                        if (ok) scores(i, j + 1);
                    }
                }
                if (!ok) break;
                mma_commit(&bars->empty[(2 * j + 1) % STAGES]);
                if (j + 1 < all) mma_commit(&bars->empty[(2 * j + 2) % STAGES]);
            }
            volatile int never = 0;
            mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, &never, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax, one row a thread
        const int i = warp >> 2, quad = warp & 3;
        const int n = steps[i];
        const int row = first_row + i * PT + quad * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t t_s = tmem + lanes + i * PT, t_o = tmem + lanes + 2 * PT + i * D;
        const int lim = row + off;                              // the last key the row sees
        const float sl2 = p.scale_log2, raise = RAISE / sl2;
        float m = -INFINITY, l = 0.0f;
        uint32_t scans = 0;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = warp_wait(&bars->s_full[i], j & 1, abort, I8R_DEV_TMEM_TIMEOUT);
            if (!ok) break;
            tc_fence_after_sync();
            // a step that every row of the tile sees whole needs no mask
            const bool cut = j * PT + PT - 1 > first_row + i * PT + off;
            const int seen = lim - j * PT;                      // columns 0 .. seen stay
            // The scores are read twice (tensor memory's bandwidth is idle
            // otherwise), so that half of them are in registers at a time.
            float x[2][32];
            auto fetch = [&](int h) {
                uint32_t r[2][32];
                tmem_ld32(t_s + 64 * h, r[0]);
                tmem_ld32(t_s + 64 * h + 32, r[1]);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 64; ++e) x[e >> 5][e & 31] = __uint_as_float(r[e >> 5][e & 31]);
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        x[e >> 5][e & 31] = 64 * h + e <= seen ? x[e >> 5][e & 31] : -INFINITY;
                }
            };
            float mx = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                fetch(h);
                float top[4] = {mx, x[0][0], x[0][1], x[0][2]};
#pragma unroll
                for (int e = 3; e < 63; e += 2)
                    top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], x[e >> 5][e & 31], x[(e + 1) >> 5][(e + 1) & 31]);
                mx = fmaxf(max3(top[0], top[1], top[2]), fmaxf(top[3], x[1][31]));
            }
            if (__any_sync(0xFFFFFFFFu, mx > m + raise)) {
                const float to = fmaxf(m, mx);
                const float alpha = m == -INFINITY ? 0.0f : ex2((m - to) * sl2);
                l *= alpha;
                m = to;
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
            // p = 2^(x * scale_log2 - m * scale_log2); a row that has seen nothing yet has all -inf
            const float ref = m == -INFINITY ? 0.0f : -m * sl2;
            const uint64_t sl22 = pack2(sl2, sl2), ref2 = pack2(ref, ref);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                fetch(h);
                uint32_t out[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 y = unpack2(fma2(pack2(x[e >> 4][2 * (e & 15)], x[e >> 4][2 * (e & 15) + 1]), sl22, ref2));
                    const float p0 = ex2(y.x), p1 = ex2(y.y);
                    sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                    const __half2 h2 = __floats2half2_rn(p0, p1);
                    out[e] = *reinterpret_cast<const uint32_t *>(&h2);
                }
                tmem_st32(t_s + 32 * h, out);
            }
            const float2 s2 = unpack2(add2(sum[0], sum[1]));
            l += s2.x + s2.y;
            tmem_wait_st();
            if (cut) {
                // V's rows of a step that a mask cuts: this warp looks at 32 of them
                const int k = 2 * j + 1;
                uint8_t *v = ring + k % STAGES * Shape::TILE_BYTES;
                ok = warp_wait(&bars->full[k % STAGES], (k / STAGES) & 1, abort, I8R_DEV_PIPELINE_TIMEOUT);
                if (!ok) break;
                bool bad = false;
#pragma unroll
                for (int c = 0; c < Shape::CHUNKS; ++c)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        bad |= not_finite(*reinterpret_cast<const uint4 *>(v + c * Shape::CHUNK_BYTES + quad * 4096 +
                                                                           e * 512 + lane * 16));
                if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) *static_cast<volatile int *>(&bars->dirty_step[i]) = j;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->scan[i]);
                ok = warp_wait(&bars->scan[i], scans & 1, abort, I8R_DEV_TMEM_TIMEOUT);
                if (!ok) break;
                ++scans;
                if (*static_cast<volatile int *>(&bars->dirty_step[i]) == j) {
                    // P V over the keys that the row sees
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                        if (j > 0) {
                            tmem_ld32(t_o + 32 * c, o);
                            tmem_wait_ld();
                        }
#pragma unroll 1
                        for (int kk = 0; kk < PT; kk += 2) {
                            uint32_t pp;
                            tmem_ld1(t_s + kk / 2, pp);
                            tmem_wait_ld();
                            const float2 pf = __half22float2(*reinterpret_cast<const __half2 *>(&pp));
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                if (j * PT + kk + z > lim) continue;
                                const float pz = z ? pf.y : pf.x;
                                const uint8_t *src = v + (c >> 1) * Shape::CHUNK_BYTES + (kk + z) * 128;
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    const uint4 q = *reinterpret_cast<const uint4 *>(src + (((4 * (c & 1) + u) ^ ((kk + z) & 7)) << 4));
                                    const __half2 *hv = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float2 f = __half22float2(hv[e]);
                                        uint32_t &o0 = o[8 * u + 2 * e], &o1 = o[8 * u + 2 * e + 1];
                                        o0 = __float_as_uint(fmaf(pz, f.x, __uint_as_float(o0)));
                                        o1 = __float_as_uint(fmaf(pz, f.y, __uint_as_float(o1)));
                                    }
                                }
                            }
                            __syncwarp();
                        }
                        tmem_st32(t_o + 32 * c, o);
                    }
                    tmem_wait_st();
                    if (lane == 0) *static_cast<volatile int *>(&bars->skip_step[i]) = j;
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_ready[i]);
        }
        if (ok && n > 0) {
            ok = warp_wait(&bars->o_full[i], 0, abort, I8R_DEV_TMEM_TIMEOUT);
            tc_fence_after_sync();
        }
        if (ok) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            __half *dst = p.O + static_cast<size_t>(qr.x + row) * p.ldo + static_cast<size_t>(head) * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(t_o + 32 * c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                uint4 out[4];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const __half2 h2 = __floats2half2_rn(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    reinterpret_cast<uint32_t *>(out)[e] = *reinterpret_cast<const uint32_t *>(&h2);
                }
                // a row that sees no key: zeros, whatever its tile's steps left
                if (lim < 0) out[0] = out[1] = out[2] = out[3] = make_uint4(0u, 0u, 0u, 0u);
                if (row < nq) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * e) = out[e];
                }
            }
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

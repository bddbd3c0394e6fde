// Attention of single tokens over the 8-bit key/value cache.
//
// For query head q of sequence b (key/value head h = q / G):
//   x_t = scale * (sK/127) * sum_d Q[d] Kc[t,d]          t < len
//   O   = sum_t e^(x_t - max x) * (sV/127) * Vc[t,:] / sum_t e^(x_t - max x)
// in one pass over the codes with a running maximum and sum.
//
// Bound by reading the codes from HBM once (2 D bytes a token and head), so the
// work is cut by bytes: a step is 16 tokens of one (sequence, key/value head,
// tile of 8*NT queries), all steps of the call in order are dealt to the warps of
// a persistent grid in equal contiguous ranges, and every warp works through its
// range alone.  A range usually begins and ends inside an item; those pieces are
// merged per CTA in shared memory, and the few items that cross CTAs by
// combine_kernel from at most two pieces a CTA, always in the same order.
//
// The codes travel by cp.async into slots that only the copying lane reads (the
// ring is the lanes' registers, spilled: no barrier, no bank conflict, and three
// steps in flight for a 16-warp SM are about 128 KB), laid out so that a lane
// gets its own mma.sync fragments: m16n8k16 with tokens (then values' columns) as
// the 16 rows and queries as the 8 columns, which suits one to eight queries per
// head; at under one MMA per 10 cycles the legacy tensor path is nowhere near a
// limit.  Codes become fp16 exactly (byte permutes against 0x6400 and one
// subtraction), scores and sums are fp32, and p = e^(x - max) <= 1 is rounded to
// fp16 (2^-11) for the second product, below the rounding of the fp16 output.
#pragma once

#include "device_common.cuh"
#include "gemm_decode.cuh"
#include "kv_cache.cuh"

namespace i8r {
namespace attn {

constexpr int STEP = 16;                 // tokens per step
constexpr int DEC_WARPS = 8;
constexpr int DEC_THREADS = 32 * DEC_WARPS;
constexpr int DEC_MAX_CTAS = 320;        // of the persistent grid (two per SM), which sizes the workspace

struct DecodeParams {
    kv::Cache c;
    const __half *Q;
    __half *O;
    long long ldq, ldo;
    const int32_t *lengths;
    int B, G, GT, tile;                  // queries per kv head, tiles of `tile` queries per kv head
    float scale_log2;                    // scale * log2(e)
    float *part;                         // [2 * CTAs][tile][D + 2]
    int stages;
};

// Bytes of one warp's ring stage: 16 tokens of K and V, and the two scales.
__host__ __device__ constexpr int stage_bytes(int D) { return 2 * STEP * D + 16; }
// Floats of one piece: maximum, sum and D values per query.
__host__ __device__ constexpr int piece_floats(int tile, int D) { return tile * (D + 2); }
__host__ __device__ inline size_t decode_smem(int tile, int D, int stages) {
    return static_cast<size_t>(DEC_WARPS) * (static_cast<size_t>(stages) * stage_bytes(D) + piece_floats(tile, D) * 4);
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
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
// Two codes, in bytes `lo` and `hi` of x (x = codes ^ 0x80), as fp16: 0x6400 + u
// is 1024 + u, and 1024 + u - 1152 = u - 128, exactly.
template <int kSel>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t x) {
    const uint32_t u = __byte_perm(x, 0x64646464u, kSel);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
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
__device__ __forceinline__ long long steps_of(const DecodeParams &p, int b) {      // of all its items
    return static_cast<long long>((length_of(p, b) + STEP - 1) / STEP) * (p.c.H * p.GT);
}
__device__ __forceinline__ long long total_steps(const DecodeParams &p) {
    long long n = 0;
    for (int b = threadIdx.x & 31; b < p.B; b += 32) n += steps_of(p, b);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, d);
    return n;
}

// A place in the order of steps: sequence b, item hg = h*GT + query tile, step.
struct Place {
    int b, hg, step, steps, len;
    __device__ __forceinline__ void at(const DecodeParams &p, long long u) {
        long long r = 0;
        b = kv::find_item(u, p.B, &r, [&](int s) { return steps_of(p, s); });
        len = length_of(p, b);
        steps = (len + STEP - 1) / STEP;
        hg = static_cast<int>(r / steps);
        step = static_cast<int>(r % steps);
    }
    // the next step; false past the last sequence
    __device__ __forceinline__ bool next(const DecodeParams &p) {
        if (++step < steps) return true;
        step = 0;
        if (++hg < p.c.H * p.GT) return true;
        hg = 0;
        do {
            if (++b >= p.B) return false;
            len = length_of(p, b);
        } while (len == 0);
        steps = (len + STEP - 1) / STEP;
        return true;
    }
};

// The block of a place, its table entry read ahead of the step that uses it; a
// bad one (reported) reads block 0, which is always there.
__device__ __forceinline__ int page_at(const DecodeParams &p, const Place &w) {
    const int page = kv::block_of(p.c.table, p.c.max_blocks, p.c.num_blocks, w.b, w.step / (kv::BLOCK / STEP));
    return page < 0 ? 0 : page;
}

template <int D>
__device__ __forceinline__ void issue_step(const DecodeParams &p, const Place &w, int page, uint32_t slot) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const size_t at = static_cast<size_t>(page) * p.c.H + w.hg / p.GT;
    const size_t row0 = (at * kv::BLOCK + (w.step % (kv::BLOCK / STEP)) * STEP) * D;
    const int8_t *K = p.c.codes[0] + row0, *V = p.c.codes[1] + row0;
    uint32_t dst = slot + lane * 16;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < D / 64; ++c, dst += 512) cp_async_16(dst, K + (g + 8 * r) * D + 64 * c + 16 * t, 16u);
    if (D == 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k, dst += 512) cp_async_16(dst, V + (2 * t + (k & 1) + 8 * (k >> 1)) * D + 16 * g, 16u);
    } else {
        dst -= lane * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k, dst += 256) cp_async_8(dst, V + (2 * t + (k & 1) + 8 * (k >> 1)) * D + 8 * g);
    }
    if (lane < 2) cp_async_4(slot + 2 * STEP * D + 4 * lane, (lane ? p.c.scale[1] : p.c.scale[0]) + at);
}

// One piece of an item in memory: per query its maximum (log2 units), its sum
// and its D unnormalised values.
template <int D>
__device__ __forceinline__ float *piece_row(float *piece, int q) { return piece + q * (D + 2); }

template <int D, int NT>
struct State {
    float acc[D / 16][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t q[D / 16][NT][2];

    // a new item: its queries (zero past the last one), nothing summed yet
    __device__ __forceinline__ void begin(const DecodeParams &p, const Place &w) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int h = w.hg / p.GT, q0 = (w.hg % p.GT) * p.tile;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int qi = q0 + 8 * n + g;
            const bool have = qi < p.G && 8 * n + g < p.tile;
            const __half *src = p.Q + static_cast<size_t>(w.b) * p.ldq + static_cast<size_t>(h * p.G + qi) * D + 16 * t;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint2 v = have ? __ldg(reinterpret_cast<const uint2 *>(src + 64 * (k >> 2) + 4 * (k & 3)))
                                     : make_uint2(0u, 0u);
                q[k][n][0] = v.x;
                q[k][n][1] = v.y;
            }
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[k][n][e] = 0.0f;
    }

    __device__ __forceinline__ void step(const DecodeParams &p, const Place &w, const uint8_t *slot) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        const uint8_t *mine = slot + lane * 16;
        const float2 sc = *reinterpret_cast<const float2 *>(slot + 2 * STEP * D);
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
        // scores: rows are tokens g and g+8, a lane's four codes of a word are the
        // MMA's columns 2t, 2t+1, 2t+8, 2t+9 (the queries' fragments follow suit)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const uint4 r0 = *reinterpret_cast<const uint4 *>(mine + 512 * c);
            const uint4 r1 = *reinterpret_cast<const uint4 *>(mine + 512 * (D / 64 + c));
            const uint32_t a[4] = {r0.x, r0.y, r0.z, r0.w}, b[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = a[k] ^ 0x80808080u, v = b[k] ^ 0x80808080u;
                const uint32_t a0 = codes_to_half2<0x4140>(u), a2 = codes_to_half2<0x4342>(u);
                const uint32_t a1 = codes_to_half2<0x4140>(v), a3 = codes_to_half2<0x4342>(v);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(x[n], a0, a1, a2, a3, q[4 * c + k][n][0], q[4 * c + k][n][1]);
            }
        }
        const float ks = p.scale_log2 * (sc.x * (1.0f / 127.0f)), vs = sc.y * (1.0f / 127.0f);
        const int t0 = w.step * STEP + g;
        const bool in0 = t0 < w.len, in1 = t0 + 8 < w.len;
        uint32_t b0[NT], b1[NT];
        float alpha[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float u = in0 ? x[n][e] * ks : -INFINITY, v = in1 ? x[n][2 + e] * ks : -INFINITY;
                float top = fmaxf(u, v);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                top = fmaxf(top, m[n][e]);
                alpha[n][e] = ex2(m[n][e] - top);
                m[n][e] = top;
                pr[e] = ex2(u - top);
                pr[2 + e] = ex2(v - top);
                l[n][e] = fmaf(l[n][e], alpha[n][e], pr[e] + pr[2 + e]);
            }
            const __half2 h0 = __floats2half2_rn(pr[0], pr[1]), h1 = __floats2half2_rn(pr[2], pr[3]);
            b0[n] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h0));
            b1[n] = transpose8x8(*reinterpret_cast<const uint32_t *>(&h1));
        }
        // values: rows are columns d of V, two per lane and MMA; k is the token
        const uint8_t *vsrc = slot + STEP * D + lane * (D / 8);
        uint32_t v[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (D == 128) {
                const uint4 r = *reinterpret_cast<const uint4 *>(vsrc + 512 * k);
                v[k][0] = r.x, v[k][1] = r.y, v[k][D / 32 - 2] = r.z, v[k][D / 32 - 1] = r.w;
            } else {
                const uint2 r = *reinterpret_cast<const uint2 *>(vsrc + 256 * k);
                v[k][0] = r.x, v[k][1] = r.y;
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
                const uint32_t a0 = codes_to_half2<0x4140>(lo), a1 = codes_to_half2<0x4342>(lo);
                const uint32_t a2 = codes_to_half2<0x4140>(hi), a3 = codes_to_half2<0x4342>(hi);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(part, a0, a1, a2, a3, b0[n], b1[n]);
                    float(&o)[4] = acc[2 * i + half][n];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = fmaf(part[e], vs, o[e] * alpha[n][e & 1]);
                }
            }
        }
    }

    // The item's output, or its piece.
    __device__ __forceinline__ void end(const DecodeParams &p, const Place &w, bool whole, float *piece) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int h = w.hg / p.GT, q0 = (w.hg % p.GT) * p.tile;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                const int qi = 8 * n + 2 * t + e;
                if (qi >= p.tile || q0 + qi >= p.G) continue;
                if (whole) {
                    const float inv = 1.0f / sum;
                    __half2 o[D / 16];
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) o[k] = __floats2half2_rn(acc[k][n][e] * inv, acc[k][n][2 + e] * inv);
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
                            make_float2(acc[k][n][e], acc[k][n][2 + e]);
                }
            }
    }
};

// What a warp left of an item it did not do alone.
struct Piece {
    int b, hg;                           // b < 0: none
    bool starts, ends;                   // the piece holds the item's first / last step
};

template <int D, int NT>
__global__ void __launch_bounds__(DEC_THREADS, NT == 1 ? 2 : 1)
    attention_decode_kernel(const __grid_constant__ DecodeParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Piece pieces[2 * DEC_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warp_ring = p.stages * stage_bytes(D);
    uint8_t *ring = smem + warp * warp_ring;
    const uint32_t ring_u = smem_u32(ring);
    // a warp's first piece is written while its ring is still in use, its last one into the ring
    float *firsts = reinterpret_cast<float *>(smem + DEC_WARPS * warp_ring);
    if (threadIdx.x < 2 * DEC_WARPS) pieces[threadIdx.x].b = -1;
    // sequences without tokens
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (length_of(p, b) == 0)
            for (int i = threadIdx.x; i < p.c.H * p.G * (D / 8); i += DEC_THREADS)
                *reinterpret_cast<uint4 *>(p.O + static_cast<size_t>(b) * p.ldo + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();

    const long long S = total_steps(p);
    const int warps = gridDim.x * DEC_WARPS, me = blockIdx.x * DEC_WARPS + warp;
    const long long u0 = decode::unit_begin(S, me, warps), u1 = decode::unit_begin(S, me + 1, warps);
    if (u0 < u1) {
        Place w, ahead;
        w.at(p, u0);
        ahead = w;
        long long issued = u0;
        int page = page_at(p, ahead);
        int fill = 0;
        auto issue = [&]() {
            if (issued < u1) {
                issue_step<D>(p, ahead, page, ring_u + fill * stage_bytes(D));
                if (++issued < u1) {
                    ahead.next(p);
                    page = page_at(p, ahead);
                }
            }
            cp_async_commit();
            if (++fill == p.stages) fill = 0;
        };
        for (int s = 0; s + 1 < p.stages; ++s) issue();
        State<D, NT> st;
        st.begin(p, w);
        bool starts = w.step == 0, first = true;
        int slot = 0;
        for (long long u = u0; u < u1; ++u) {
            if (p.stages == 2)
                cp_async_wait<0>();
            else if (p.stages == 3)
                cp_async_wait<1>();
            else
                cp_async_wait<2>();
            __syncwarp();                       // lanes 0 and 1 copied the scales; the slot read last is free
            issue();
            st.step(p, w, ring + slot * stage_bytes(D));
            if (++slot == p.stages) slot = 0;
            const bool ends = w.step + 1 == w.steps;
            if (ends || u + 1 == u1) {
                const bool whole = starts && ends;
                if (!whole) {
                    if (!first) {
                        cp_async_wait<0>();     // nothing of the ring is in flight or unread
                        __syncwarp();
                    }
                    if (lane == 0) pieces[2 * warp + (first ? 0 : 1)] = Piece{w.b, w.hg, starts, ends};
                }
                st.end(p, w, whole, first ? firsts + warp * piece_floats(p.tile, D) : reinterpret_cast<float *>(ring));
                first = false;
                if (u + 1 < u1) {
                    w.next(p);
                    st.begin(p, w);
                    starts = true;
                }
            } else {
                w.next(p);
            }
        }
    }
    __syncthreads();

    // Merge this CTA's pieces, item by item in order; an item that begins or ends
    // in another CTA leaves one piece for combine_kernel, in slot 0 if it begins
    // where the CTA's range does, else in slot 1.
    const long long U0 = decode::unit_begin(S, blockIdx.x * DEC_WARPS, warps);
    for (int i = 0; i < 2 * DEC_WARPS;) {
        const Piece a = pieces[i];
        if (a.b < 0) {
            ++i;
            continue;
        }
        int j = i + 1, last = i;
        for (; j < 2 * DEC_WARPS; ++j) {
            if (pieces[j].b < 0) continue;
            if (pieces[j].b != a.b || pieces[j].hg != a.hg) break;
            last = j;
        }
        const bool whole = a.starts && pieces[last].ends;
        const int first_warp = blockIdx.x * DEC_WARPS + (i >> 1);
        const int out_slot = ((i & 1) == 0 && decode::unit_begin(S, first_warp, warps) == U0) ? 0 : 1;
        float *out = p.part + static_cast<size_t>(2 * blockIdx.x + out_slot) * piece_floats(p.tile, D);
        const int h = a.hg / p.GT, q0 = (a.hg % p.GT) * p.tile;
        const int nq = min(p.tile, p.G - q0);
        for (int e = threadIdx.x; e < nq * (D / 2); e += DEC_THREADS) {
            const int q = e / (D / 2), d = 2 * (e % (D / 2));
            float top = -INFINITY;
            for (int k = i; k <= last; ++k) {
                if (pieces[k].b < 0) continue;
                float *src = (k & 1) ? reinterpret_cast<float *>(smem + (k >> 1) * warp_ring)
                                     : firsts + (k >> 1) * piece_floats(p.tile, D);
                top = fmaxf(top, piece_row<D>(src, q)[0]);
            }
            float sum = 0.0f;
            float2 o = make_float2(0.0f, 0.0f);
            for (int k = i; k <= last; ++k) {
                if (pieces[k].b < 0) continue;
                float *src = (k & 1) ? reinterpret_cast<float *>(smem + (k >> 1) * warp_ring)
                                     : firsts + (k >> 1) * piece_floats(p.tile, D);
                const float *row = piece_row<D>(src, q);
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
}

// The items that cross CTAs.  Block (c, q): if the range of CTA c + 1 begins
// inside an item that began in CTA c's range, that item's query q is the sum of
// the pieces of CTAs c, c + 1, ... up to the one where it ends.  One thread per
// value; the pieces are read in order, eight ahead.
template <int D>
__global__ void __launch_bounds__(D) attention_combine_kernel(const __grid_constant__ DecodeParams p, int ctas) {
    griddep_wait();
    const int c = blockIdx.x, q = blockIdx.y, d = threadIdx.x;
    const long long S = total_steps(p);
    const int warps = ctas * DEC_WARPS;
    auto begin = [&](int cta) { return decode::unit_begin(S, cta * DEC_WARPS, warps); };
    const long long u = begin(c + 1);
    if (u >= S || u == begin(c)) return;
    Place w;
    w.at(p, u);
    const long long start = u - w.step, end = start + w.steps;
    const int q0 = (w.hg % p.GT) * p.tile;
    if (w.step == 0 || start < begin(c) || q0 + q >= p.G) return;
    const int last = decode::unit_owner(S, end - 1, warps) / DEC_WARPS;
    auto row = [&](int cta) {
        const int slot = start <= begin(cta) ? 0 : 1;
        return piece_row<D>(p.part + static_cast<size_t>(2 * cta + slot) * piece_floats(p.tile, D), q);
    };
    float top = -INFINITY, sum = 0.0f, o = 0.0f;
    for (int k0 = c; k0 <= last; k0 += 8) {
        float m[8], l[8], v[8], was = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] = -INFINITY;
            l[k] = v[k] = 0.0f;
            // a CTA without steps (fewer steps than warps) has no piece
            if (k0 + k <= last && begin(k0 + k) < begin(k0 + k + 1)) {
                const float *r = row(k0 + k);
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
    const int h = w.hg / p.GT;
    p.O[static_cast<size_t>(w.b) * p.ldo + static_cast<size_t>(h * p.G + q0 + q) * D + d] = __float2half_rn(o / sum);
}

}  // namespace attn
}  // namespace i8r

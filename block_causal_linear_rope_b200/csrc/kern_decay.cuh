// Decayed linear attention on the CUDA cores: prompts in fp32 arithmetic, and
// the single-token step of both types.
#pragma once

#include "decay.cuh"

namespace blin {

// ---------------------------------------------------------------------------- prompts
constexpr int kSimtChunk = 64;

template <int D>
struct SimtCfg {
    static constexpr int C = kSimtChunk, P = D + 4;  // rows padded by 16 bytes: no bank conflicts on 16-byte reads
    static constexpr int PP = C + 4;
    static constexpr int FLOATS = 4 * C * P + C * PP + D * P + C + 4;
    static constexpr int BYTES = FLOATS * 4;
};

// V consecutive floats of shared memory, 16 bytes at a time, the second 16 bytes `far` floats on.
template <int V>
__device__ __forceinline__ void lds_vec(const float *p, int far, float (&f)[V]) {
    if constexpr (V == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        f[0] = v.x, f[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(p + far * i);
            f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
        }
    }
}

// One segment of one fp32 head, 64 tokens at a time:
//   o_i = scale (sum_{j <= i} g^{i-j} (q_i . k_j) v_j + g^{i+1} q_i S),
//   S  <- g^n S + sum_j (g^{n-1-j} k_j)^T v_j.
// 16 x 16 threads hold a 4 x 4 tile of the scores, 4 x D/16 of the outputs and
// D/16 x D/16 of the state.  The state's values stay in registers and a copy in
// shared memory feeds the products; the keys are stored twice, plain and
// weighted, so that a chunk needs three barriers: tiles written, scores
// written, tiles read.  Everything is an fp32 FMA: bf16 or tf32 parts of fp32
// operands would need six tensor products to keep this accuracy.  Bound: shared
// memory reads (60% of their peak) and FMA issue (40%).
// STATES: local states only (phase 1).
template <int D, bool STATES>
__global__ void __launch_bounds__(256) decay_simt_kernel(const DecayArgs a) {
    using Cfg = SimtCfg<D>;
    constexpr int C = Cfg::C, P = Cfg::P, PP = Cfg::PP, W = D / 16;
    constexpr int FAR = 64, X0 = W <= 4 ? W : 4;  // a thread's columns: X0 tx and, at D = 128, 64 + 4 tx
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4), *sk = sq + C * P, *sv = sk + C * P, *sw = sv + C * P, *sp = sw + C * P,
          *ss = sp + C * PP, *pw = ss + D * P;  // sw: weighted keys; pw[n] = g^n, n <= C
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int per = STATES ? a.nseg - 1 : a.nseg;
    const int bh = blockIdx.x / per, seg = blockIdx.x - bh * per;
    const int b = bh / a.H, h = bh - b * a.H;
    const int slot = decay_slot(a, b);
    const int L = slot < 0 ? 0 : decay_len(a, b);
    const int begin = seg * a.seg, end = min(begin + a.seg, L);
    const float lg = decay_log(a.log_decay, h);
    float *wsp = a.ws + (size_t)bh * a.nseg * D * D;
    float *pool = a.S && slot >= 0 ? a.S + ((size_t)slot * a.H + h) * D * D : nullptr;
    if (tid <= C) pw[tid] = decay_pow(lg, (float)tid);
    auto col = [&](int w) { return X0 * tx + (w < 4 ? w : FAR + w - 4); };
    float st[W][W];  // state rows ty * W + r, columns col(w)
#pragma unroll
    for (int r = 0; r < W; ++r)
#pragma unroll
        for (int w = 0; w < W; ++w) st[r][w] = 0.f;
    if (STATES) {
        if (seg == 0)  // the second launch may overwrite the pool while others still read the entering state
            for (int i = tid; i < D * D / 4; i += 256)
                reinterpret_cast<float4 *>(wsp)[i] =
                    pool ? reinterpret_cast<const float4 *>(pool)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    } else if (begin < L) {
        if (a.nseg == 1) {
            if (pool)
#pragma unroll
                for (int r = 0; r < W; ++r)
#pragma unroll
                    for (int w = 0; w < W; ++w) st[r][w] = pool[(ty * W + r) * D + col(w)];
        } else {
            for (int s = 0; s <= seg; ++s) {
                const float f = decay_pow(lg, (float)(begin - s * a.seg));
#pragma unroll
                for (int r = 0; r < W; ++r)
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        st[r][w] = fmaf(f, wsp[(size_t)s * D * D + (ty * W + r) * D + col(w)], st[r][w]);
            }
        }
    }
    const float *qp = static_cast<const float *>(a.q) + b * a.lq.batch + h * a.lq.head;
    const float *kp = static_cast<const float *>(a.k) + b * a.lk.batch + h * a.lk.head;
    const float *vp = static_cast<const float *>(a.v) + b * a.lv.batch + h * a.lv.head;
    float *op = static_cast<float *>(a.o) + b * a.lo.batch + h * a.lo.head;
    const DecaySplit whole(lg, (float)C);
    // acc += A rows (4 ty ...) x B, over `kend` columns of A
    auto product = [&](const float *A, int lda, const float *Bm, int kend, float (&acc)[4][W]) {
        for (int j = 0; j < kend; j += 4) {
            float av[4][4];
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) lds_vec<4>(A + (4 * ty + ii) * lda + j, 0, av[ii]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float bv[W];
                lds_vec<W>(Bm + (j + u) * P + X0 * tx, FAR, bv);
#pragma unroll
                for (int ii = 0; ii < 4; ++ii)
#pragma unroll
                    for (int w = 0; w < W; ++w) acc[ii][w] = fmaf(av[ii][u], bv[w], acc[ii][w]);
            }
        }
    };
    for (int n0 = begin; n0 < end; n0 += C) {
        const int n = min(C, end - n0);  // tokens of this chunk
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < C * (D / 4); i += 256) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            auto get = [&](const float *src, long long tok) {
                return r < n ? *reinterpret_cast<const float4 *>(src + (long long)(n0 + r) * tok + c) : zero;
            };
            const float4 k = get(kp, a.lk.tok), v = get(vp, a.lv.tok);
            const float f = pw[max(n - 1 - r, 0)];
            *reinterpret_cast<float4 *>(sv + r * P + c) = v;
            *reinterpret_cast<float4 *>(sw + r * P + c) = make_float4(f * k.x, f * k.y, f * k.z, f * k.w);
            if (!STATES) {
                *reinterpret_cast<float4 *>(sk + r * P + c) = k;
                *reinterpret_cast<float4 *>(sq + r * P + c) = get(qp, a.lq.tok);
            }
        }
        if (!STATES) {
#pragma unroll
            for (int r = 0; r < W; ++r)
#pragma unroll
                for (int w = 0; w < W; ++w) ss[(ty * W + r) * P + col(w)] = st[r][w];
        }
        __syncthreads();
        if (!STATES) {
            // a warp's rows end at 8 warp + 7: columns past them are masked and skipped
            const int jmax = 8 * (tid >> 5) + 8;
            float acc[4][4];
#pragma unroll
            for (int ii = 0; ii < 4; ++ii)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) acc[ii][jj] = 0.f;
#pragma unroll 2
            for (int c = 0; c < D; c += 4) {
                float qv[4][4];
#pragma unroll
                for (int ii = 0; ii < 4; ++ii) lds_vec<4>(sq + (4 * ty + ii) * P + c, 0, qv[ii]);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    if (16 * jj < jmax) {
                        float kv[4];
                        lds_vec<4>(sk + (tx + 16 * jj) * P + c, 0, kv);
#pragma unroll
                        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
                            for (int u = 0; u < 4; ++u) acc[ii][jj] = fmaf(qv[ii][u], kv[u], acc[ii][jj]);
                    }
                }
            }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                for (int ii = 0; ii < 4; ++ii) {
                    const int i = 4 * ty + ii, j = tx + 16 * jj;
                    sp[i * PP + j] = j <= i ? acc[ii][jj] * pw[i - j] : 0.f;
                }
            float out[4][W];
#pragma unroll
            for (int ii = 0; ii < 4; ++ii)
#pragma unroll
                for (int w = 0; w < W; ++w) out[ii][w] = 0.f;
            product(sq, P, ss, D, out);
#pragma unroll
            for (int ii = 0; ii < 4; ++ii)
#pragma unroll
                for (int w = 0; w < W; ++w) out[ii][w] *= pw[4 * ty + ii + 1];
            __syncthreads();
            product(sp, PP, sv, jmax, out);
#pragma unroll
            for (int ii = 0; ii < 4; ++ii) {
                const int i = 4 * ty + ii;
                if (i < n) {
                    float *dst = op + (long long)(n0 + i) * a.lo.tok;
#pragma unroll
                    for (int w = 0; w < W; ++w) dst[col(w)] = a.scale * out[ii][w];
                }
            }
        }
        // state: the chunk's decay and its tokens
        DecaySplit g = whole;
        if (n < C) g = DecaySplit(lg, (float)n);
        float add[W][W];
#pragma unroll
        for (int r = 0; r < W; ++r)
#pragma unroll
            for (int w = 0; w < W; ++w) add[r][w] = 0.f;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            float kv[W], vv[W];
            lds_vec<W>(sw + j * P + ty * W, 4, kv);
            lds_vec<W>(sv + j * P + X0 * tx, FAR, vv);
#pragma unroll
            for (int r = 0; r < W; ++r)
#pragma unroll
                for (int w = 0; w < W; ++w) add[r][w] = fmaf(kv[r], vv[w], add[r][w]);
        }
#pragma unroll
        for (int r = 0; r < W; ++r)
#pragma unroll
            for (int w = 0; w < W; ++w) st[r][w] = fmaf(st[r][w], g.hi, fmaf(st[r][w], g.lo, add[r][w]));
    }
    if (STATES || (pool && begin < L && end == L)) {
        float *dst = STATES ? wsp + (size_t)(seg + 1) * D * D : pool;
#pragma unroll
        for (int r = 0; r < W; ++r)
#pragma unroll
            for (int w = 0; w < W; ++w) dst[(ty * W + r) * D + col(w)] = st[r][w];
    }
    if (!STATES) {  // rows past the prompt's end are zeros
        const int z0 = max(begin, L), z1 = min(begin + a.seg, a.N);
        for (long long i = tid; i < (long long)(z1 - z0) * (D / 4); i += 256) {
            const int r = (int)(i / (D / 4)), c = (int)(i - (long long)r * (D / 4)) * 4;
            *reinterpret_cast<float4 *>(op + (long long)(z0 + r) * a.lo.tok + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
}

// ---------------------------------------------------------------------------- one token
// decay_slot by each warp for itself.
__device__ __forceinline__ int decay_slot_warp(const DecayArgs &a, int b, int s, int lane) {
    if (a.slot_of == nullptr || s < 0) return s;
    int twice = 0;
    if (s < a.slots)
        for (int i = lane; i < b; i += 32) twice |= __ldg(a.slot_of + i) == s;
    twice = __any_sync(~0u, twice);
    if (s < a.slots && !twice) return s;
    if (lane == 0) atomicCAS(a.wd, 0, s >= a.slots ? WD_SLOT_RANGE : WD_SLOT_TWICE);
    return -1;
}

// A unit is 32 columns of one head's state; a thread takes 8 rows of 4 of them,
// so that the whole piece is in flight at once, and each element is read and
// written once.  Splitting by columns leaves nothing to add up between CTAs; at
// d = 128 whole rows in one CTA of 512 threads took 108 us where this takes 86
// (128 rows of 32 heads).  Bound: HBM (8 d^2 bytes per head); that call moves
// 537 MB at 6.2 TB/s.
template <int D>
struct StepCfg {
    static constexpr int CX = 8, RG = D / 8, TPU = CX * RG;  // column and row groups, threads per unit
    static constexpr int THREADS = 128, UPB = THREADS / TPU, PER = D / 32;  // units per CTA, per head
};
template <int D, typename T>
__global__ void __launch_bounds__(StepCfg<D>::THREADS) decay_step_kernel(const DecayArgs a) {
    using Cf = StepCfg<D>;
    constexpr int CX = Cf::CX, RG = Cf::RG, WPU = Cf::TPU / 32;  // warps of a unit
    __shared__ float4 part[Cf::THREADS / 32][CX];
    const int tid = threadIdx.x % Cf::TPU, lane = threadIdx.x & 31, cx = tid % CX, rg = tid / CX;
    const long long u = (long long)blockIdx.x * Cf::UPB + threadIdx.x / Cf::TPU;
    const bool there = u < (long long)a.B * a.H * Cf::PER;
    const int bh = there ? (int)(u / Cf::PER) : 0, b = bh / a.H, h = bh - b * a.H;
    const int c0 = 32 * (int)(u % Cf::PER) + 4 * cx;
    // the state's loads go out before the check for repeated slots: an entry in range is safe to read
    int s = there ? a.slot_of ? __ldg(a.slot_of + b) : b : -1;
    const bool in = s >= 0 && s < a.slots;
    float *sp = a.S + ((size_t)(in ? s : 0) * a.H + h) * D * D + c0;
    float4 st[8];
    if (in)
#pragma unroll
        for (int r = 0; r < 8; ++r) st[r] = *reinterpret_cast<const float4 *>(sp + (rg + RG * r) * D);
    s = decay_slot_warp(a, b, s, lane);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (s >= 0) {
        const T *qp = static_cast<const T *>(a.q) + b * a.lq.batch + h * a.lq.head;
        const T *kp = static_cast<const T *>(a.k) + b * a.lk.batch + h * a.lk.head;
        const T *vp = static_cast<const T *>(a.v) + b * a.lv.batch + h * a.lv.head + c0;
        const DecayMul mul(decay_log(a.log_decay, h), 1.f);
        float v[4], k[8], q[8];
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = static_cast<float>(vp[w]);
#pragma unroll
        for (int r = 0; r < 8; ++r) k[r] = static_cast<float>(kp[rg + RG * r]), q[r] = static_cast<float>(qp[rg + RG * r]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float x[4] = {st[r].x, st[r].y, st[r].z, st[r].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                x[w] = fmaf(k[r], v[w], mul(x[w]));
                acc[w] = fmaf(q[r], x[w], acc[w]);
            }
            *reinterpret_cast<float4 *>(sp + (rg + RG * r) * D) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    // row groups: those of a warp, then the unit's warps
#pragma unroll
    for (int o = CX; o < 32; o *= 2)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[w] += __shfl_xor_sync(~0u, acc[w], o);
    float4 t = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if constexpr (WPU > 1) {
        if (lane < CX) part[threadIdx.x / 32][lane] = t;
        __syncthreads();
        if (rg == 0) {
            const int w0 = threadIdx.x / Cf::TPU * WPU;
            t = part[w0][cx];
#pragma unroll
            for (int w = 1; w < WPU; ++w) {
                const float4 x = part[w0 + w][cx];
                t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
            }
        }
    }
    if (rg == 0 && there) {
        T *op = static_cast<T *>(a.o) + b * a.lo.batch + h * a.lo.head + c0;
        op[0] = static_cast<T>(a.scale * t.x);
        op[1] = static_cast<T>(a.scale * t.y);
        op[2] = static_cast<T>(a.scale * t.z);
        op[3] = static_cast<T>(a.scale * t.w);
    }
}

}  // namespace blin

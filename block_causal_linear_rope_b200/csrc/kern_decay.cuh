// Decayed linear attention: fp32 prompts, and the single-token step of both types.
#pragma once

#include "decay.cuh"

namespace blin {

// ---------------------------------------------------------------------------- prompts
constexpr int kF32Chunk = 64;

template <int D>
struct F32Cfg {
    static constexpr int C = kF32Chunk;
    // row pitches in floats: an operand read along its rows wants 4 (mod 32), one read down its columns 8, so
    // that the 32 lanes of a fragment load hit 32 banks
    static constexpr int PR = D + 4, PC = D + 8, PP = C + 4;
    static constexpr int FLOATS = 2 * C * PR + 2 * C * PC + D * PC + C * PP + C + 4;
    static constexpr int BYTES = FLOATS * 4;
    static constexpr int CTAS = D == 128 ? 1 : D == 64 ? 2 : 3;  // per SM
    // warps of a D x D product: rows x columns, and 16 x 8 tiles of a warp
    static constexpr int SM = D == 32 ? 2 : 4, SN = 8 / SM, MT = D / (16 * SM), NT = D / (8 * SN);
    static constexpr int OT = D / 16;  // tiles of a warp's outputs (16 rows x D/2 columns)
};

// x as hi + lo with hi rounded to tf32 (10 fraction bits) and lo the exact rest, of which the tensor core
// drops what is below 2^-21 of x.
__device__ __forceinline__ void split_tf32(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// acc += A (16 rows, `kend` columns) x B (`kend` rows, 8 N columns) by one warp, tiles n < live only.
// AT: A is stored with its columns as rows; BT: B is.  The tensor core rounds its running sums towards zero;
// the two small products have sums of their own, so that the large one's see one rounding per 8 columns, and
// three products in a row go to different sums.
template <int N, bool AT, bool BT>
__device__ __forceinline__ void f32_product(const float *A, int pa, const float *B, int pb, int kend, float (&acc)[N][4],
                                            int live) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float small[N][4] = {};
#pragma unroll 2
    for (int k = 0; k < kend; k += 8) {
        uint32_t ah[4], al[4], bh[N][2], bl[N][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = g + 8 * (i & 1), c = k + t + 4 * (i >> 1);
            split_tf32(AT ? A[c * pa + r] : A[r * pa + c], ah[i], al[i]);
        }
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < live)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = k + t + 4 * i, c = 8 * n + g;
                    split_tf32(BT ? B[c * pb + r] : B[r * pb + c], bh[n][i], bl[n][i]);
                }
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < live) mma_tf32(acc[n], ah, bh[n]);
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < live) mma_tf32(small[n], al, bh[n]);
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (n < live) mma_tf32(small[n], ah, bl[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += small[n][i];
}

// One segment of one fp32 head, 64 tokens at a time:
//   o_i = scale (sum_{j <= i} g^{i-j} (q_i . k_j) v_j + g^{i+1} q_i S),
//   S  <- g^n S + sum_j (g^{n-1-j} k_j)^T v_j.
// fp32 has no tensor product of its own, and FMAs alone bound the chunk at 6700
// cycles of a whole SM (d = 64; an FMA form took 177 us for 2 x 16 heads of 4000
// tokens, this one 132, with the tensor cores and the issue slots half busy).  Each
// operand is split in registers into two tf32 parts as it is read from shared
// memory, and three products (hi hi + hi lo + lo hi) keep 21 bits of it: what is
// dropped is below 2^-21 a term, unbiased, where the sums' own rounding is 2^-22
// to 2^-21.  A chunk's state product is summed from zero and added to the
// decayed state, which stays in fp32 registers, by FMAs: the tensor core rounds
// its running sums towards zero, and a long-lived state must not collect that.
// Eight warps share each product; the keys are stored twice, plain and weighted,
// so that a chunk needs three barriers.  STATES: local states only (phase 1).
template <int D, bool STATES>
__global__ void __launch_bounds__(256, F32Cfg<D>::CTAS) decay_f32_kernel(const DecayArgs a) {
    using Cfg = F32Cfg<D>;
    constexpr int C = Cfg::C, PR = Cfg::PR, PC = Cfg::PC, PP = Cfg::PP, MT = Cfg::MT, NT = Cfg::NT, OT = Cfg::OT;
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4), *sk = sq + C * PR, *sv = sk + C * PR, *sw = sv + C * PC, *ss = sw + C * PC,
          *sp = ss + D * PC, *pw = sp + C * PP;  // sw: weighted keys; ss: the entering state; pw[n] = g^n, n <= C
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t2 = 2 * (lane & 3);
    const int per = STATES ? a.npiece : a.nseg, span = STATES ? a.piece : a.seg;
    const int run = blockIdx.x / per, seg = blockIdx.x - run * per;
    const int at = run / a.H, h = run - at * a.H, b = STATES ? at : decay_row(a, at, sq), bh = STATES ? run : b * a.H + h;
    const int slot = decay_slot(a, b);
    const int L = slot < 0 ? 0 : decay_len(a, b);
    const int begin = seg * span, end = min(begin + span, L);
    const float lg = decay_log(a.log_decay, h);
    float *wsp = a.ws + (size_t)bh * (1 + a.npiece) * D * D;
    float *pool = a.S && slot >= 0 ? a.S + ((size_t)slot * a.H + h) * D * D : nullptr;
    if (tid <= C) pw[tid] = decay_pow(lg, (float)tid);
    // this warp's part of the state: element (m, n, i) is row srow + 16 m + 8 (i >> 1), column scol + 8 n + (i & 1)
    const int s0 = 16 * MT * (warp / Cfg::SN), s1 = 8 * NT * (warp % Cfg::SN), srow = s0 + g4, scol = s1 + t2;
    float st[MT][NT][4];
    auto each = [&](auto &&f) {  // pairs of neighbouring columns
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; i += 2) f(srow + 16 * m + 4 * i, scol + 8 * n, st[m][n][i], st[m][n][i + 1]);
    };
    each([&](int, int, float &x, float &y) { x = y = 0.f; });
    if (STATES) {
        if (seg == 0)  // the second launch may overwrite the pool while others still read the entering state
            for (int i = tid; i < D * D / 4; i += 256)
                reinterpret_cast<float4 *>(wsp)[i] =
                    pool ? reinterpret_cast<const float4 *>(pool)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    } else if (begin < L) {
        auto add = [&](const float *src, float f) {
            each([&](int r, int c, float &x, float &y) {
                const float2 v = *reinterpret_cast<const float2 *>(src + r * D + c);
                x = fmaf(f, v.x, x), y = fmaf(f, v.y, y);
            });
        };
        if (a.nseg > 1)
            for (int p = 0; p * a.piece <= begin; ++p) add(wsp + (size_t)p * D * D, decay_pow(lg, (float)(begin - p * a.piece)));
        else if (pool) add(pool, 1.f);
    }
    const float *qp = static_cast<const float *>(a.q) + b * a.lq.batch + h * a.lq.head;
    const float *kp = static_cast<const float *>(a.k) + b * a.lk.batch + h * a.lk.head;
    const float *vp = static_cast<const float *>(a.v) + b * a.lv.batch + h * a.lv.head;
    float *op = static_cast<float *>(a.o) + b * a.lo.batch + h * a.lo.head;
    const DecaySplit whole(lg, (float)C);
    const int wr = warp >> 1, wc = warp & 1, i0 = 16 * wr + g4;  // scores and outputs: 4 x 2 warps, rows i0 and i0 + 8
    for (int n0 = begin; n0 < end; n0 += C) {
        const int n = min(C, end - n0);  // tokens of this chunk
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < C * (D / 4); i += 256) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            auto get = [&](const float *src, long long tok) {
                return r < n ? *reinterpret_cast<const float4 *>(src + (long long)(n0 + r) * tok + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            const float4 k = get(kp, a.lk.tok), v = get(vp, a.lv.tok);
            const float f = pw[max(n - 1 - r, 0)];
            *reinterpret_cast<float4 *>(sv + r * PC + c) = v;
            *reinterpret_cast<float4 *>(sw + r * PC + c) = make_float4(f * k.x, f * k.y, f * k.z, f * k.w);
            if (!STATES) {
                *reinterpret_cast<float4 *>(sk + r * PR + c) = k;
                *reinterpret_cast<float4 *>(sq + r * PR + c) = get(qp, a.lq.tok);
            }
        }
        if (!STATES)
            each([&](int r, int c, float &x, float &y) { *reinterpret_cast<float2 *>(ss + r * PC + c) = make_float2(x, y); });
        // the next chunk's rows on their way into L2 while this one is multiplied
        for (int i = tid; i < C * (D / 32); i += 256) {
            const int r = n0 + C + i / (D / 32), c = i % (D / 32) * 32;
            if (r < end) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(kp + (long long)r * a.lk.tok + c));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(vp + (long long)r * a.lv.tok + c));
                if (!STATES) asm volatile("prefetch.global.L2 [%0];" ::"l"(qp + (long long)r * a.lq.tok + c));
            }
        }
        __syncthreads();
        if (!STATES) {
            // a warp's rows end at 16 wr + 15: columns past them are masked, and whole tiles of them skipped
            float p[4][4] = {};
            f32_product<4, false, true>(sq + 16 * wr * PR, PR, sk + 32 * wc * PR, PR, D, p, 2 * wr + 2 - 4 * wc);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const int r = i0 + 4 * i, c = 32 * wc + 8 * u + t2;
                    *reinterpret_cast<float2 *>(sp + r * PP + c) =
                        make_float2(c <= r ? p[u][i] * pw[r - c] : 0.f, c + 1 <= r ? p[u][i + 1] * pw[r - c - 1] : 0.f);
                }
            float out[OT][4] = {};
            f32_product<OT, false, false>(sq + 16 * wr * PR, PR, ss + D / 2 * wc, PC, D, out, OT);
#pragma unroll
            for (int u = 0; u < OT; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[u][i] *= pw[i0 + 8 * (i >> 1) + 1];
            __syncthreads();
            f32_product<OT, false, false>(sp + 16 * wr * PP, PP, sv + D / 2 * wc, PC, 16 * wr + 16, out, OT);
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (i0 + 4 * i < n) {
                    float *dst = op + (long long)(n0 + i0 + 4 * i) * a.lo.tok + D / 2 * wc + t2;
#pragma unroll
                    for (int u = 0; u < OT; ++u)
                        *reinterpret_cast<float2 *>(dst + 8 * u) = make_float2(a.scale * out[u][i], a.scale * out[u][i + 1]);
                }
        }
        // state: the chunk's decay and its tokens
        DecaySplit g = whole;
        if (n < C) g = DecaySplit(lg, (float)n);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float add[NT][4] = {};
            f32_product<NT, true, false>(sw + s0 + 16 * m, PC, sv + s1, PC, (n + 7) & ~7, add, NT);
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) st[m][u][i] = fmaf(st[m][u][i], g.hi, fmaf(st[m][u][i], g.lo, add[u][i]));
        }
    }
    if (STATES || (pool && begin < L && end == L)) {
        float *dst = STATES ? wsp + (size_t)(seg + 1) * D * D : pool;
        each([&](int r, int c, float &x, float &y) { *reinterpret_cast<float2 *>(dst + r * D + c) = make_float2(x, y); });
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
// decay_slot by each warp for itself.  Row b looks at b slots: 256 bytes a warp in
// the mean of 128 rows, beside its 4 KB of state; as much as the state (though from
// the caches) at 2000 rows.
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

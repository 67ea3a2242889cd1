// Shared declarations of the decayed linear attention (blin_decay_*): the
// arguments of one call, the decay arithmetic, and the launchers.
//
// A prompt is cut into `nseg` segments of whole chunks.  With one segment a CTA
// walks a head's prompt from its cached state to its end.  With more, a first
// launch reduces every segment but the last, in pieces of one or several to a
// segment, to their local states (what a piece's tokens add to a zero state), and a
// second one walks the segments side by side, each from the sum of the states
// before it:
//   S_in(s) = g^{start_s} S_0 + sum over the pieces p before it of g^{start_s - end_p} local(p).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "blin_internal.cuh"

namespace blin {

struct DecayArgs {
    const void *q, *k, *v;
    void *o;
    Layout lq, lk, lv, lo;
    int B, H, N;
    const float *log_decay;  // [H]
    float scale;
    const int *lengths;  // [B] or NULL
    float *S;            // [slots][H][d][d] or NULL
    int slots;
    const int *slot_of;  // [B] or NULL
    bool sorted;         // blocks take the batch rows longest first (B <= kMaxSorted)
    int nseg, seg;       // segments of a prompt and tokens per segment (whole chunks)
    int npiece, piece;   // nseg > 1: pieces of all segments but the last and tokens per piece (whole chunks)
    float *ws;           // nseg > 1: [B*H][1 + npiece][d*d]: the entering state, then the pieces' local states
    int *wd;
};

// A head's log decay as the kernels use it: at most 0, NaN where the caller's
// entry is positive or NaN.  The floor keeps -inf * 0 tokens at a power of 1;
// exp(-10000 n) is 0 in fp32 for every n >= 1.
__device__ __forceinline__ float decay_log(const float *log_decay, int h) {
    const float x = __ldg(log_decay + h);
    return x <= 0.f ? fmaxf(x, -1e4f) : __int_as_float(0x7fc00000);
}

// g^n = exp(lg * n).  The product's rounding error is recovered by an FMA and
// applied to first order: the exponent of a far token is exact to fp32, where
// expf(lg * n) alone would lose |lg n| * 2^-24.
__device__ __forceinline__ float decay_pow(float lg, float n) {
    const float p = lg * n;
    if (!(p > -150.f)) return p <= -150.f ? 0.f : p;  // underflow, or NaN
    const float e = expf(p);
    return fmaf(e, fmaf(lg, n, -p), e);
}

// One state element decayed by g = e^lgn: S * g as S + S (g - 1) while g is near
// 1, where rounding g itself would be repeated at every step and add up.
struct DecayMul {
    float m;
    bool near;
    __device__ __forceinline__ DecayMul(float lg, float n) {
        const float p = lg * n;
        near = p > -0.5f;
        if (near) {
            const float e = expm1f(p);
            m = fmaf(e + 1.f, fmaf(lg, n, -p), e);
        } else {
            m = decay_pow(lg, n);
        }
    }
    __device__ __forceinline__ float operator()(float s) const { return near ? fmaf(s, m, s) : s * m; }
};

// g^n as the sum of an fp32 value and the rest, so that a state multiplied by it at
// every chunk does not collect the same rounding error of g^n each time.
struct DecaySplit {
    float hi, lo;
    __device__ __forceinline__ DecaySplit(float lg, float n) {
        const DecayMul m(lg, n);
        hi = m.near ? 1.f + m.m : m.m;
        lo = m.near ? (1.f - hi) + m.m : 0.f;
    }
};

// The pool slot of batch row b, -1 when the row is idle (all threads of the
// block call it).  An entry out of range, or one that an earlier row has, makes
// the row idle and is recorded in the watchdog word.
__device__ __forceinline__ int decay_slot(const DecayArgs &a, int b) {
    if (a.slot_of == nullptr) return b;
    const int s = __ldg(a.slot_of + b);
    int twice = 0;
    if (s >= 0 && s < a.slots)
        for (int i = threadIdx.x; i < b; i += blockDim.x) twice |= __ldg(a.slot_of + i) == s;
    twice = __syncthreads_or(twice);
    if (s < 0) return -1;
    if (s >= a.slots || twice) {
        if (threadIdx.x == 0) atomicCAS(a.wd, 0, s >= a.slots ? WD_SLOT_RANGE : WD_SLOT_TWICE);
        return -1;
    }
    return s;
}

// Tokens of batch row b.
__device__ __forceinline__ int decay_len(const DecayArgs &a, int b) {
    return a.lengths ? min(max(__ldg(a.lengths + b), 0), a.N) : a.N;
}

// The batch row that the blocks of run i take (in the launch that makes the outputs;
// all threads of the block call it).  Rows of unequal lengths go longest first, idle
// ones last, ties by index: blocks start in the order of their numbers, and a long
// row that started last would run on alone (8 x 32 heads of up to 2048 tokens,
// d = 128: 124 us by index, 95 longest first).  With many rows the ends even out by
// themselves and the ranks cost each block more: 100 x 16 heads of up to 512 bf16
// tokens, d = 64, take 123 us by index and 137 longest first, of up to 1024, d = 128,
// 353 and 359 (fp32, 512 tokens, would gain: 358 and 313).
constexpr int kMaxSorted = 64;
static __device__ __noinline__ int sorted_row(const int *lengths, const int *slot_of, int B, int N, int i, int *len) {
    const int t = threadIdx.x;
    if (t < B) len[t] = slot_of && __ldg(slot_of + t) < 0 ? 0 : min(max(__ldg(lengths + t), 0), N);
    __syncthreads();
    if (t < B) {
        int rank = 0;
        const int own = len[t];
#pragma unroll 4
        for (int r = 0; r < B; ++r) rank += len[r] + (r < t) > own;
        if (rank == i) len[kMaxSorted] = t;
    }
    __syncthreads();
    return len[kMaxSorted];
}
// scratch: kMaxSorted + 1 ints of shared memory that nobody writes before the block's next barrier
__device__ __forceinline__ int decay_row(const DecayArgs &a, int i, void *scratch) {
    if (!a.sorted) return i;
    // the same in every lane, as the compiler then knows too
    return __shfl_sync(~0u, sorted_row(a.lengths, a.slot_of, a.B, a.N, i, static_cast<int *>(scratch)), 0);
}

// Prompts: fp32 in tf32 parts (kern_decay.cuh), bf16 on tcgen05 (kern_decay_tc.cuh).
cudaError_t launch_decay_f32(const DecayArgs &a, int d, cudaStream_t s);
cudaError_t launch_decay_tc(const DecayArgs &a, int d, cudaStream_t s);
cudaError_t launch_decay_step(const DecayArgs &a, int d, bool bf16, cudaStream_t s);

}  // namespace blin

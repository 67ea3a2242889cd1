// Decayed linear attention: argument checks, the split of a prompt into
// segments, and the launches of blin_decay_prefill and blin_decay_step.
#include <algorithm>
#include <cmath>

#include "kern_decay.cuh"
#include "kern_decay_tc.cuh"

namespace blin {

// Raises a kernel's dynamic shared-memory limit (once per context and kernel).
template <auto Kernel>
static cudaError_t allow_smem(int bytes) {
    static ContextCache<int> done;
    const unsigned long long ctx = current_context_id();
    int have = 0;
    if (done.get(ctx, &have) && have >= bytes) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.put(ctx, bytes);
    return e;
}

// A prompt's launches: with several segments the local states first.
template <auto States, auto Outputs, typename... Args>
static cudaError_t launch_prompt(const DecayArgs &a, int states_threads, int states_smem, int threads, int smem,
                                 cudaStream_t s, const Args &...args) {
    cudaError_t e = cudaSuccess;
    if (a.nseg > 1) {
        if ((e = allow_smem<States>(states_smem)) != cudaSuccess) return e;
        States<<<(unsigned)(a.B * a.H * a.npiece), states_threads, states_smem, s>>>(args..., a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        note_launch();
    }
    if ((e = allow_smem<Outputs>(smem)) != cudaSuccess) return e;
    Outputs<<<(unsigned)(a.B * a.H * a.nseg), threads, smem, s>>>(args..., a);
    if ((e = cudaGetLastError()) == cudaSuccess) note_launch();
    return e;
}

template <int D>
static cudaError_t f32(const DecayArgs &a, cudaStream_t s) {
    constexpr int smem = F32Cfg<D>::BYTES;
    return launch_prompt<decay_f32_kernel<D, true>, decay_f32_kernel<D, false>>(a, 256, smem, 256, smem, s);
}

cudaError_t launch_decay_f32(const DecayArgs &a, int d, cudaStream_t s) {
    return d == 32 ? f32<32>(a, s) : d == 64 ? f32<64>(a, s) : f32<128>(a, s);
}

// The warpgroups that take more registers draw on what the kernel was launched with: a build with fewer
// than planned would leave them waiting, so it is not launched.
template <auto Kernel>
static bool has_registers(int n) {
    static ContextCache<int> cache;
    const unsigned long long ctx = current_context_id();
    int have = 0;
    if (!cache.get(ctx, &have)) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, Kernel) != cudaSuccess) return false;
        cache.put(ctx, have = at.numRegs);
    }
    return have >= n;
}

template <int D>
static cudaError_t tc(const DecayArgs &a, const DecayMaps &m, cudaStream_t s) {
    using CS = DecayTc<D, true>;
    using CO = DecayTc<D, false>;
    if (CO::RSPLIT && !has_registers<decay_tc_kernel<D, false>>(CO::RL)) return cudaErrorInvalidConfiguration;
    if (CS::RSPLIT && !has_registers<decay_tc_kernel<D, true>>(CS::RL)) return cudaErrorInvalidConfiguration;
    return launch_prompt<decay_tc_kernel<D, true>, decay_tc_kernel<D, false>>(a, CS::THREADS, CS::BYTES, CO::THREADS,
                                                                             CO::BYTES, s, m);
}

cudaError_t launch_decay_tc(const DecayArgs &a, int d, cudaStream_t s) {
    DecayMaps m;
    if (!make_map4(&m.q, a.q, a.lq, a.B, a.H, a.N, d, 128, &m.swap_q) ||
        !make_map4(&m.k, a.k, a.lk, a.B, a.H, a.N, d, 128, &m.swap_k) ||
        !make_map4(&m.v, a.v, a.lv, a.B, a.H, a.N, d, 128, &m.swap_v) ||
        !make_map4(&m.o, a.o, a.lo, a.B, a.H, a.N, d, 32, &m.swap_o))
        return cudaErrorInvalidValue;
    return d == 32 ? tc<32>(a, m, s) : d == 64 ? tc<64>(a, m, s) : tc<128>(a, m, s);
}

template <int D, typename T>
static cudaError_t step(const DecayArgs &a, cudaStream_t s) {
    using Cf = StepCfg<D>;
    const long long units = (long long)a.B * a.H * Cf::PER;
    decay_step_kernel<D, T><<<(unsigned)((units + Cf::UPB - 1) / Cf::UPB), Cf::THREADS, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) note_launch();
    return e;
}

cudaError_t launch_decay_step(const DecayArgs &a, int d, bool bf16, cudaStream_t s) {
    switch (d) {
        case 32: return bf16 ? step<32, __nv_bfloat16>(a, s) : step<32, float>(a, s);
        case 64: return bf16 ? step<64, __nv_bfloat16>(a, s) : step<64, float>(a, s);
        default: return bf16 ? step<128, __nv_bfloat16>(a, s) : step<128, float>(a, s);
    }
}

}  // namespace blin

using namespace blin;

static bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Segments of a prompt and their pieces.  A launch runs its units in waves over the
// SMs, so its time goes as waves x (chunks of a unit + what a unit costs besides); a
// split prompt has a first launch (states only) with cheaper chunks, and its second
// one's units add up the states before them.  The split with the smallest sum is
// taken, from sizes alone.  The costs are in chunks of the path's second launch
// as measured on a B200 with all SMs full: a chunk of 128 bf16 tokens takes 2.0 to
// 3.1 us at d = 32 (two CTAs to an SM), 2.0 to 2.7 at d = 64 and 4.6 to 5.0 at
// d = 128, one of 64 fp32 tokens 8 us at d = 32 (three CTAs), 12 at d = 64 (two; one
// alone 7) and 19 at d = 128, and a launch and a unit's start a few us either way
// (4 heads of 300 fp32 tokens: 39 us in one piece, 19 in five; 16 heads of 1024
// bf16 tokens, d = 64: 23 us in one, 21 in four).
//   kMaxStates: a unit of the second launch adds up the states before it one after
// the other, which the cost `join` states too low to hold for many of them.  One
// head of 40000 tokens with at most 16, 32, 48 and 64 states: 164, 145, 160 and
// 160 us at d = 128, 73, 53, 49 and 48 at d = 64 in bf16; 399, 211, 159 and 127 in
// fp32 at d = 64, which has the most to gain from more.
//   kMaxPieces: 32 heads of 32768 bf16 tokens, d = 128, take 440, 431, 404 and 404
// us with at most 1, 2, 4 and 8 pieces to a segment.
//   kSms: a part with fewer SMs gets a worse split, not a wrong one.
static constexpr int kSms = 148, kMaxStates = 32, kMaxPieces = 4;
struct Split {
    int nseg, seg, npiece, piece;
};
struct SplitCosts {
    double unit, join, chunk1, unit1, launch1;  // a unit's start, a state it adds, a chunk, a unit's start and the rest of the first launch
};
static Split split_prompt(long long heads, int N, int chunk, int resident, const SplitCosts &k) {
    const int nc = std::max(1, (N + chunk - 1) / chunk);
    const long long slots = (long long)kSms * resident;
    const auto waves = [&](long long units) { return (double)((units + slots - 1) / slots); };
    Split best{1, nc * chunk, 0, nc * chunk};
    double cost = waves(heads) * (nc + k.unit);
    for (int s = 2; s <= std::min(nc, kMaxStates); ++s)
        for (int m = 1; m <= kMaxPieces && (s - 1) * m < kMaxStates; ++m) {
            const int plen = (nc + s * m - 1) / (s * m), len = plen * m, n = (nc + len - 1) / len;
            if (n != s || heads * n * m >= (1LL << 31)) continue;
            const int pieces = (n - 1) * m;
            const double t = waves(heads * n) * (len + k.unit + k.join * pieces) +
                             waves(heads * pieces) * (k.chunk1 * plen + k.unit1) + k.launch1;
            if (t < cost) {
                cost = t;
                best = Split{n, len * chunk, pieces, plen * chunk};
            }
            if (heads * pieces >= 4 * slots) break;
        }
    return best;
}

// Blocks of the second launch that an SM holds.
static int resident(int d, blin_dtype dt) {
    if (dt == BLIN_BF16) return d == 32 ? 2 : 1;
    return d == 128 ? F32Cfg<128>::CTAS : d == 64 ? F32Cfg<64>::CTAS : F32Cfg<32>::CTAS;
}

static Split split_of(int B, int H, int N, int d, blin_dtype dt) {
    const long long heads = (long long)B * H;
    if (dt == BLIN_BF16) return split_prompt(heads, N, 128, resident(d, dt), {2.0, 0.25, d == 128 ? 0.67 : 0.5, 1.5, 1.5});
    return split_prompt(heads, N, kF32Chunk, resident(d, dt), {0.3, 0.05, 0.4, 0.3, 0.3});
}

static size_t workspace_of(const Split &sp, int B, int H, int d) {
    return sp.nseg > 1 ? sizeof(float) * (size_t)B * H * (1 + sp.npiece) * d * d : 16;
}

static blin_status check_shape(int B, int H, int N, int d, blin_dtype dt) {
    if (B < 1 || H < 1 || N < 0) return failf(BLIN_ERR_INVALID_ARG, "B and H must be >= 1 and N >= 0 (got %d, %d, %d)", B, H, N);
    if (d != 32 && d != 64 && d != 128) return failf(BLIN_ERR_SHAPE, "head dim d must be 32, 64 or 128 (got %d)", d);
    if (dt != BLIN_F32 && dt != BLIN_BF16) return failf(BLIN_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if ((long long)B * H >= (1LL << 24) || N >= (1 << 30))
        return failf(BLIN_ERR_SHAPE, "problem too large (B*H = %lld, N = %d)", (long long)B * H, N);
    return BLIN_OK;
}

// Everything a prefill and a step check alike; fills the call's arguments.
static blin_status check_call(DecayArgs &a, const void *q, const void *k, const void *v, void *o, blin_dtype dt, int B,
                              int H, int N, int d, const float *log_decay, float scale, const blin_decay_layouts *lay,
                              float *S, int slots, const int *slot_of) {
    blin_status rc = check_shape(B, H, N, d, dt);
    if (rc != BLIN_OK) return rc;
    if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || log_decay == nullptr)
        return failf(BLIN_ERR_INVALID_ARG, "q, k, v, o and log_decay must be non-NULL device pointers");
    if (!std::isfinite(scale)) return failf(BLIN_ERR_INVALID_ARG, "scale must be finite");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(S, 16))
        return failf(BLIN_ERR_ALIGN, "q, k, v, o and S must be 16-byte aligned");
    if (!aligned(log_decay, 4) || !aligned(slot_of, 4))
        return failf(BLIN_ERR_ALIGN, "log_decay, lengths and slot_of_row must be 4-byte aligned");
    if (S != nullptr && slots < 1) return failf(BLIN_ERR_STATE, "slots must be >= 1 (got %d)", slots);
    if (S != nullptr && slot_of == nullptr && slots != B)
        return failf(BLIN_ERR_STATE, "without slot_of_row the pool holds one slot per row: slots = %d, B = %d", slots, B);
    if (S == nullptr && slot_of != nullptr) return failf(BLIN_ERR_STATE, "slot_of_row needs a state pool");
    if (static_cast<const void *>(o) == q || static_cast<const void *>(o) == k || static_cast<const void *>(o) == v)
        return failf(BLIN_ERR_INVALID_ARG, "o must not overlap q, k or v");
    a = DecayArgs{};
    const char *name[4] = {"q", "k", "v", "o"};
    Layout *to[4] = {&a.lq, &a.lk, &a.lv, &a.lo};
    for (int i = 0; i < 4; ++i) {
        blin_layout l;
        if (lay) {
            l = (&lay->q)[i];
            if (N <= 1) l.token = d;  // a single token never moves
        }
        if ((rc = get_layout(lay ? &l : nullptr, B, H, N, d, dt, name[i], to[i])) != BLIN_OK) return rc;
    }
    a.q = q, a.k = k, a.v = v, a.o = o;
    a.B = B, a.H = H, a.N = N;
    a.log_decay = log_decay;
    a.scale = scale;
    a.S = S;
    a.slots = slots;
    a.slot_of = slot_of;
    return BLIN_OK;
}

static blin_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? BLIN_OK : failf(BLIN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

extern "C" {

size_t blin_decay_workspace_size(int B, int H, int N, int d, blin_dtype dt) {
    if (check_shape(B, H, N, d, dt) != BLIN_OK) return 0;
    return workspace_of(split_of(B, H, N, d, dt), B, H, d);
}

blin_status blin_decay_prefill(const void *q, const void *k, const void *v, void *o, blin_dtype dt, int B, int H, int N,
                               int d, const float *log_decay, float scale, const blin_decay_layouts *layouts,
                               const int *lengths, float *S, int slots, const int *slot_of_row, void *workspace,
                               size_t ws_bytes, blin_stream stream) {
    const TraceRange trace("blin_decay_prefill");
    DecayArgs a;
    blin_status rc = check_call(a, q, k, v, o, dt, B, H, N, d, log_decay, scale, layouts, S, slots, slot_of_row);
    if (rc != BLIN_OK) return rc;
    if (!aligned(lengths, 4)) return failf(BLIN_ERR_ALIGN, "log_decay, lengths and slot_of_row must be 4-byte aligned");
    if (N == 0) return BLIN_OK;
    const Split sp = split_of(B, H, N, d, dt);
    const size_t need = workspace_of(sp, B, H, d);
    if (sp.nseg > 1 && (workspace == nullptr || ws_bytes < need))
        return failf(BLIN_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", workspace ? ws_bytes : 0, need);
    if (!aligned(workspace, 16)) return failf(BLIN_ERR_ALIGN, "workspace must be 16-byte aligned");
    a.lengths = lengths;
    a.nseg = sp.nseg;
    a.seg = sp.seg;
    a.npiece = sp.npiece;
    a.piece = sp.piece;
    // the order of rows matters where not all blocks start at once
    a.sorted = lengths != nullptr && B > 1 && B <= kMaxSorted && (long long)B * H * sp.nseg > kSms * resident(d, dt);
    a.ws = static_cast<float *>(workspace);
    if ((a.wd = watchdog_ptr()) == nullptr) return failf(BLIN_ERR_CUDA, "no CUDA device");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(dt == BLIN_BF16 ? launch_decay_tc(a, d, s) : launch_decay_f32(a, d, s), "decayed attention launch");
}

blin_status blin_decay_step(const void *q, const void *k, const void *v, void *o, blin_dtype dt, int B, int H, int d,
                            const float *log_decay, float scale, const blin_decay_layouts *layouts, float *S, int slots,
                            const int *slot_of_row, blin_stream stream) {
    const TraceRange trace("blin_decay_step");
    DecayArgs a;
    if (S == nullptr) return failf(BLIN_ERR_INVALID_ARG, "a step needs a state pool");
    const blin_status rc = check_call(a, q, k, v, o, dt, B, H, 1, d, log_decay, scale, layouts, S, slots, slot_of_row);
    if (rc != BLIN_OK) return rc;
    if ((a.wd = watchdog_ptr()) == nullptr) return failf(BLIN_ERR_CUDA, "no CUDA device");
    return launched(launch_decay_step(a, d, dt == BLIN_BF16, static_cast<cudaStream_t>(stream)), "decay step launch");
}

}  // extern "C"

// Rotary embedding over the axes (t, y, x), forward and inverse, of q and k in
// one launch: pairs (2j, 2j+1) of each axis section turn by p * theta^(-2j/d_axis).
//
// Bound: HBM (each element read and written once, 3 flops each).  A thread owns
// one 16-byte piece of a token's row, computes the angles of its pairs once into
// registers, and walks the heads with them: an angle costs one evaluation per
// token and pair and CTA instead of one per head, and the loads of several heads
// are in flight at a time.
//
// Angles: the frequency of a pair, in turns per position, is computed on the
// host in double precision and handed over as a kernel argument; position x
// frequency is reduced to a fraction of a turn in double precision, and the sine
// and cosine of that fraction are taken in fp32.  A position of 2^31 keeps an
// angle error of 2^31 * 2^-53 turns; fp32 angles would be off by 1e-2 radians at
// a position of 1e5 already.
//
// Measured on a B200: q and k of 70 heads of 75600 tokens, d = 32, bf16: 219 us, 94%
// of the rate of a plain copy; 2 x 48 heads of 4099 fp32 tokens, d = 64: 37 us, the
// time of a copy.  A single token of 64 requests (40 heads, d = 128) takes 6.0 us
// in a graph, nearly all of it one thread's way through positions, angles and one
// round of loads, and 6.5 us of host time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "blin_internal.cuh"

namespace {

using blin::Layout;

constexpr int kMaxPairs = 128;
constexpr int kThreads = 256;
constexpr long long kCtas = 8 * 148;  // eight on every SM

struct RopeArgs {
    const void *in[2];
    void *out[2];
    Layout li[2], lo[2];
    int heads[2];         // q's and k's
    int B, N, d;
    int tile, side;       // tokens per CTA, and heads it takes at a time
    int hsplit;           // CTAs that share a run of tokens, by heads
    int pairs, py, px;    // rotated pairs; first pair of the y and x sections
    int HW, Wg, t0;       // grid positions
    const int *pos;       // given positions or NULL
    int shared_pos;
    float sign;
    double freq[kMaxPairs];  // turns per position
};

__device__ __forceinline__ float2 turn(const RopeArgs &a, int b, int n, int p) {
    const int axis = p < a.py ? 0 : p < a.px ? 1 : 2;
    int at;
    if (a.pos) {
        at = __ldg(a.pos + ((a.shared_pos ? 0LL : (long long)b * a.N) + n) * 3 + axis);
    } else {
        const int f = n / a.HW, r = n - f * a.HW, y = r / a.Wg;
        at = axis == 0 ? a.t0 + f : axis == 1 ? y : r - y * a.Wg;
    }
    const double x = (double)at * a.freq[p];
    const float fr = (float)(x - rint(x));
    float s, c;
    sincospif(2.f * fr, &s, &c);
    return make_float2(c, a.sign * s);
}

// 16 bytes: 4 fp32 (2 pairs) or 8 bf16 (4 pairs)
__device__ __forceinline__ uint32_t rotate_bf16(uint32_t w, float2 cs) {
    const float x = __uint_as_float(w << 16), y = __uint_as_float(w & 0xFFFF0000u);
    const __nv_bfloat162 h = __floats2bfloat162_rn(fmaf(x, cs.x, -y * cs.y), fmaf(x, cs.y, y * cs.x));
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
struct Piece {
    static constexpr int VN = 16 / (int)sizeof(T), VP = VN / 2;  // elements and pairs
    float2 cs[VP];
    int left;  // pairs to rotate; those past the last section's end are copied bit for bit
    __device__ __forceinline__ uint4 rotate(uint4 v) const {
        if constexpr (sizeof(T) == 2) {
            if (left > 0) v.x = rotate_bf16(v.x, cs[0]);
            if (left > 1) v.y = rotate_bf16(v.y, cs[1]);
            if (left > 2) v.z = rotate_bf16(v.z, cs[2]);
            if (left > 3) v.w = rotate_bf16(v.w, cs[3]);
        } else {
            const float x = __uint_as_float(v.x), y = __uint_as_float(v.y), z = __uint_as_float(v.z), w = __uint_as_float(v.w);
            if (left > 0) {
                v.x = __float_as_uint(fmaf(x, cs[0].x, -y * cs[0].y));
                v.y = __float_as_uint(fmaf(x, cs[0].y, y * cs[0].x));
            }
            if (left > 1) {
                v.z = __float_as_uint(fmaf(z, cs[1].x, -w * cs[1].y));
                v.w = __float_as_uint(fmaf(z, cs[1].y, w * cs[1].x));
            }
        }
        return v;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    using P = Piece<T>;
    constexpr int U = 8;  // heads in flight per thread
    const int vecs = a.d / P::VN, per = a.tile * vecs;
    const int tiles = (a.N + a.tile - 1) / a.tile;
    const int hs = blockIdx.x % a.hsplit, bt = blockIdx.x / a.hsplit;
    const int b = bt / tiles;
    const int hh = threadIdx.x / per, e = threadIdx.x - hh * per, r = e / vecs, j = e - r * vecs;
    const int n = (bt - b * tiles) * a.tile + r;
    if (hh >= a.side || n >= a.N) return;
    P piece;
    piece.left = a.pairs - j * P::VP;
#pragma unroll
    for (int i = 0; i < P::VP; ++i)
        piece.cs[i] = i < piece.left ? turn(a, b, n, j * P::VP + i) : make_float2(1.f, 0.f);
    const int all = a.heads[0] + a.heads[1];
    const int h0 = (int)((long long)all * hs / a.hsplit), h1 = (int)((long long)all * (hs + 1) / a.hsplit);
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const int first = w ? a.heads[0] : 0;
        int h = max(h0 - first, 0) + hh;
        const int end = min(h1 - first, a.heads[w]);
        const T *in = static_cast<const T *>(a.in[w]) + b * a.li[w].batch + n * a.li[w].tok + j * P::VN;
        T *out = static_cast<T *>(a.out[w]) + b * a.lo[w].batch + n * a.lo[w].tok + j * P::VN;
        const long long si = a.li[w].head, so = a.lo[w].head;
        for (; h < end; h += U * a.side) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * a.side < end) v[u] = *reinterpret_cast<const uint4 *>(in + (h + u * a.side) * si);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u * a.side < end) *reinterpret_cast<uint4 *>(out + (h + u * a.side) * so) = piece.rotate(v[u]);
        }
    }
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" blin_status blin_rope(const void *q, void *q_out, int Hq, const void *k, void *k_out, int Hk, blin_dtype dt,
                                 int B, int N, int d, const blin_geom *g, int t0, const int *positions, int shared,
                                 int inverse, const blin_rope_layouts *layouts, blin_stream stream) {
    using blin::failf;
    const blin::TraceRange trace("blin_rope");
    if (g == nullptr) return failf(BLIN_ERR_INVALID_ARG, "geom is NULL");
    if (q == nullptr || q_out == nullptr || (k == nullptr) != (k_out == nullptr))
        return failf(BLIN_ERR_INVALID_ARG, "q and q_out must be non-NULL device pointers, k and k_out both or neither");
    if (dt != BLIN_F32 && dt != BLIN_BF16) return failf(BLIN_ERR_DTYPE, "unknown dtype %d", (int)dt);
    if (B < 1 || N < 0 || Hq < 1 || (k && Hk < 1))
        return failf(BLIN_ERR_INVALID_ARG, "B, Hq and Hk must be >= 1 and N >= 0 (got %d, %d, %d, %d)", B, Hq, Hk, N);
    if (d < 8 || d > 2 * kMaxPairs || d % 8) return failf(BLIN_ERR_SHAPE, "d must be a multiple of 8 up to 256 (got %d)", d);
    if ((inverse != 0 && inverse != 1) || (shared != 0 && shared != 1))
        return failf(BLIN_ERR_INVALID_ARG, "inverse and shared must be 0 or 1");
    int sum = 0;
    for (int ax = 0; ax < 3; ++ax) {
        const int n = g->rope_split[ax];
        if (n < 0 || n > d || (n & 1)) return failf(BLIN_ERR_SHAPE, "rope_split entries must be even, >= 0 and at most d");
        sum += n;
    }
    if (sum > d) return failf(BLIN_ERR_SHAPE, "rope_split sums to %d, more than d = %d", sum, d);
    if (!(g->theta > 0.f) || !std::isfinite(g->theta)) return failf(BLIN_ERR_INVALID_ARG, "theta must be finite and > 0");
    RopeArgs a = {};
    if (positions == nullptr) {
        if (g->T < 0 || g->Hgt < 1 || g->Wid < 1 || t0 < 0)
            return failf(BLIN_ERR_INVALID_ARG, "T and t0 must be >= 0, Hgt and Wid >= 1");
        const long long hw = (long long)g->Hgt * g->Wid;
        if (hw > (1 << 30) || (long long)g->T * hw != N)
            return failf(BLIN_ERR_SHAPE, "N = %d but T*Hgt*Wid = %lld", N, (long long)g->T * hw);
        if ((long long)t0 + g->T >= (1LL << 30)) return failf(BLIN_ERR_SHAPE, "frame index overflow");
        a.HW = (int)hw;
        a.Wg = g->Wid;
        a.t0 = t0;
    }
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16) || !aligned(positions, 4))
        return failf(BLIN_ERR_ALIGN, "q, k and the outputs must be 16-byte aligned, positions 4-byte aligned");
    const int all = Hq + (k ? Hk : 0);
    if (N >= (1 << 30) || (long long)B * all >= (1LL << 24)) return failf(BLIN_ERR_SHAPE, "problem too large");
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int heads[2] = {Hq, k ? Hk : 0};
    for (int w = 0; w < 2; ++w) {
        if (!heads[w]) continue;
        blin_layout l[2];
        for (int i = 0; i < 2 && layouts; ++i) {
            l[i] = (&layouts->q)[2 * w + i];
            if (N <= 1) l[i].token = d;  // a single token never moves
        }
        blin_status rc;
        if ((rc = blin::get_layout(layouts ? &l[0] : nullptr, B, heads[w], N, d, dt, w ? "k" : "q", &a.li[w])) != BLIN_OK ||
            (rc = blin::get_layout(layouts ? &l[1] : nullptr, B, heads[w], N, d, dt, w ? "k_out" : "q_out", &a.lo[w])) !=
                BLIN_OK)
            return rc;
        const Layout &x = a.li[w], &y = a.lo[w];
        if (in[w] == out[w] && (x.tok != y.tok || x.head != y.head || x.batch != y.batch))
            return failf(BLIN_ERR_SHAPE, "an output in place of its input must have its strides");
        a.in[w] = in[w];
        a.out[w] = out[w];
        a.heads[w] = heads[w];
    }
    if (N == 0) return BLIN_OK;
    a.B = B;
    a.N = N;
    a.d = d;
    a.pos = positions;
    a.shared_pos = shared;
    a.sign = inverse ? -1.f : 1.f;
    a.py = g->rope_split[0] / 2;
    a.px = a.py + g->rope_split[1] / 2;
    a.pairs = sum / 2;
    for (int ax = 0, p = 0; ax < 3; ++ax)
        for (int j = 0; j < g->rope_split[ax] / 2; ++j, ++p)
            a.freq[p] = std::pow((double)g->theta, -2.0 * j / g->rope_split[ax]) * 0.15915494309189533577;
    // As many tokens as fill a CTA with one head's pieces, and several heads side by side where the call has
    // fewer; heads are split over CTAs until there are kCtas, or each has one round of loads.
    const int vecs = d * (dt == BLIN_BF16 ? 2 : 4) / 16;
    a.tile = std::max(1, std::min(kThreads / vecs, N));
    a.side = std::min(all, kThreads / (a.tile * vecs));
    const long long runs = (long long)B * ((N + a.tile - 1) / a.tile);
    a.hsplit = (int)std::max(1LL, std::min<long long>((kCtas + runs - 1) / runs, all / (4 * a.side)));
    if (runs * a.hsplit >= (1LL << 31)) return failf(BLIN_ERR_SHAPE, "problem too large");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(runs * a.hsplit);
    if (dt == BLIN_BF16) rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a);
    else rope_kernel<float><<<grid, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return failf(BLIN_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
    blin::note_launch();
    return BLIN_OK;
}

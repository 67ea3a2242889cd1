// Decayed linear attention of bf16 prompts on the tensor cores (sm_100a).
//
// A CTA walks one segment of one head, 128 tokens at a time.  Per chunk, with
// i, j the tokens of the chunk, n their number and g the head's decay:
//   scores   P_ij = g^{i-j} (q_i . k_j) for j <= i, else 0        (128 x 128, K = d)
//   outputs  o_i  = scale (sum_j P_ij v_j + g^{i+1} q_i S)         (128 x d, K = 128 and K = d)
//   state    S   <- g^n S + sum_j k_j^T (g^{n-1-j} v_j)            (d x d, K = 128)
// All four products run on tcgen05.mma with fp32 accumulators in TMEM.
//
// Precision.  P is rounded to bf16 (its product's other operand is bf16 already,
// and so is the result).  The S that multiplies q is handed over in two bf16
// parts, 16 bits of it: rounded once like P, the two would add as much as the
// result's own rounding does (2.35e-3 of the outputs' norm against 1.66e-3;
// with two parts 1.74e-3 for slow decays, 2.1e-3 for fast ones, where P's share
// is large), and the second part's products cost 6 to 11% of the time at d >= 64
// and nothing at d = 32.  The state itself is fp32 and stays in registers from
// chunk to chunk; the weighted values g^{n-1-j} v_j of its update are split into
// three bf16 parts (8 + 8 + 8 bits), so that its product carries fp32 accuracy
// (at most 4e-7 of the state's norm, most of it the tensor core's rounding of
// running sums towards zero).
//
// Roles: a TMA producer thread, two MMA issuing threads (scores and outputs,
// state), warpgroups that weight the scores (TMEM -> registers -> P as bf16
// in TMEM), that weight and split the values (shared memory -> shared
// memory), and that own the state and the outputs.  They hand over through
// mbarriers; every wait is bounded.
//
// Why 128 tokens: the scores fill the 128 lanes of one product.  A token then
// costs (256 + 5 d) d multiply-adds, 0.038 ns of the tensor cores at d = 64 and
// 0.12 at d = 128 (4096 a cycle and SM, 1.6 GHz), where its 8 d bytes cost the
// memory 0.08 and 0.16.  Why one
// head per CTA: the state then never leaves the registers, and K, V, Q and O
// cross the memory once.
//
// Measured on B200s, sustained (the range of three runs on different cards): 4 x
// 32 heads of 32760 tokens, d = 64: 552 to 580 us (3.7 to 3.9 TB/s); 32 heads of
// 32768, d = 128: 452 to 471 us; 70 heads of 32760, d = 32: 236 to 247 us.  What
// bounds it: a chunk takes 3700 cycles of an SM at d = 64 (about 8000 at d = 128,
// 4600 for two CTAs at d = 32), the round of score product, weights and value
// product that one score buffer allows (two, tried in an earlier form of this
// kernel, made each chunk's tiles stay longer in the landing ring: 528 us where
// that form took 511), at 37 to 44% tensor and 42 to 50% issue utilisation; and the
// card's power: it runs at its 1000 W limit at 1.55 to 1.75 GHz (a plain copy of
// random data alone takes 997 W at 6.4 TB/s), so that less work per chunk shows
// as a higher clock, not as fewer cycles.  M =
// 64 state products at d <= 64 (d = 32 repeats its 32 features by a leading byte
// offset of 0, and the threads of each copy take half of the columns) serve that.
#pragma once

#include <type_traits>

#include "decay.cuh"
#include "tc_util.cuh"

namespace blin {

template <int D, bool STATES>
struct DecayTc {
    static constexpr int C = 128;                     // tokens per chunk
    static constexpr int AW = D == 32 ? 32 : 64;      // features per swizzle atom
    static constexpr int NAT = D / AW;                // atoms per tile
    static constexpr int ROWB = 2 * AW;
    static constexpr int SUB = C * ROWB, TILE = NAT * SUB;
    static constexpr uint32_t LAYOUT = D == 32 ? 4u : 2u;  // 64B / 128B swizzle
    static constexpr int TPC = STATES ? 2 : 3;             // tiles landed per chunk: V, K (, Q)
    static constexpr int NSLOT = D == 128 ? 4 : 9;
    // weighted values: items of IT tokens, three parts each, in a ring of NVB
    static constexpr int IT = D == 128 ? 16 : D == 64 && STATES ? 32 : 64, NIT = C / IT;
    static constexpr int NVB = !STATES ? 2 : D == 128 ? 8 : D == 64 ? 4 : 2;
    static constexpr int VSUB = IT * ROWB, VPART = NAT * VSUB, VITEM = 3 * VPART;
    static constexpr int SIMG = 2 * D * D;  // a bf16 state image; there are two, high and low part
    static constexpr int OSTG = STATES || D == 128 ? 0 : TILE;      // output staging (d = 128: in the chunk's Q slot)
    // TMEM columns: scores / P, inner and carried outputs, state product.  The three parts of the values
    // multiply side by side where there is room for a column range each (KVN = 3), else the low part is
    // added to the middle one's (2), or all to one (1).
    static constexpr int KVN = D == 128 ? 1 : D == 64 || STATES ? 3 : 2, KVC = KVN * D;
    static constexpr int ZTILE = KVN == 2 ? 16 * ROWB : 0;  // 16 rows of zeros in front of the weighted values
    static constexpr int OFF_Z = NSLOT * TILE, OFF_V = OFF_Z + ZTILE, OFF_S = OFF_V + NVB * VITEM,
                         OFF_O = OFF_S + (STATES ? 0 : 2 * SIMG);
    static constexpr int OFF_CTRL = OFF_O + OSTG;
    static constexpr int NBAR = 2 * NSLOT + 2 * NVB + 13;
    static constexpr int OFF_PW = OFF_CTRL + 512;  // g^n for n = 0 .. 128, then scale g^{31 - m} for m < 32
    static constexpr int BYTES = OFF_PW + 4 * (132 + 32) + 1024;
    static_assert(8 * NBAR <= 504, "barriers");
    static_assert(BYTES <= (D == 32 ? 113 : 227) * 1024, "shared memory");
    // Warps: XG and TG warpgroups share the scores and the values of a chunk, UW warps hold the state, ZW the
    // outputs (0: the state's do both).  A d = 32 CTA has one warpgroup of each and no ZW, as two CTAs share an
    // SM.  The last warpgroup holds the producer and the MMA threads.
    static constexpr int XG = STATES ? 0 : D == 32 ? 1 : 2, TG = STATES ? (D == 32 ? 2 : 4) : D == 32 ? 1 : 2,
                         UW = D == 128 ? 8 : 4;
    static constexpr int XW = 4 * XG, TW = 4 * TG, ZW = STATES || D == 32 ? 0 : 4, OW = ZW ? ZW : UW;
    static constexpr int THREADS = 32 * (XW + TW + UW + ZW + 4);
    static constexpr int SHARE = 16, RELEASE = SHARE + 1;  // arrivals that free a landing slot
    static constexpr int KB = STATES ? 2 : 1;  // state products in TMEM
    static constexpr int KVM = D == 128 ? 128 : 64;  // rows of the state product
    static constexpr int T_OA = 128, T_OI = T_OA + D, T_KV = STATES ? 0 : T_OI + D;
    static constexpr int TCOLS = D == 32 ? 256 : STATES && D == 128 ? 256 : 512;
    static_assert(T_KV + KB * KVC <= TCOLS, "TMEM columns");
    // P: 8 columns for 16 of its own, in 64 free columns where there are (d = 64), else each in the first half
    // of the scores' columns that it was made of.
    static constexpr bool POWN = !STATES && TCOLS - (T_KV + KB * KVC) >= 64;
    static constexpr int T_P = POWN ? T_KV + KB * KVC : 0, PSTEP = POWN ? 8 : 16;
    static constexpr int NCOL = D == 128 ? 64 : D * D / 128;  // state columns per thread
    // With many warps the kernel is launched with RL registers a thread, and the warpgroups that hold the state
    // or the outputs draw on what the others give up.
    static constexpr bool RSPLIT = STATES ? D == 128 : D != 32;
    static constexpr int RL = D == 128 && !STATES ? 64 : 72;
    static constexpr int RX = !RSPLIT ? 0 : D == 128 ? 56 : 64, RT = !RSPLIT ? 0 : D == 128 && !STATES ? 48 : 56,
                         RU = !RSPLIT ? 0 : D == 64 ? 112 : STATES ? 104 : 96, RZ = !RSPLIT ? 0 : D == 128 ? 64 : 80,
                         RC = !RSPLIT ? 0 : D == 128 && !STATES ? 48 : STATES ? 56 : 72;
    static_assert(XW * RX + TW * RT + UW * RU + ZW * RZ + 4 * RC <= THREADS / 32 * RL, "registers");
};

// Maps and swaps of one call's operands.
struct DecayMaps {
    CUtensorMap q, k, v, o;
    int swap_q, swap_k, swap_v, swap_o;
};

template <int D, bool STATES>
struct DecayUnit {
    using Cf = DecayTc<D, STATES>;
    const DecayArgs &a;
    uint8_t *base;
    uint64_t *bars;
    float *pw, *lead;
    uint32_t tmem;
    int b, h, begin, end;  // tokens [begin, end) of batch row b, head h
    float lg;
    float *pool, *wsp;
    int seg;

    // Barriers: full/empty of the landing slots, ready/free of the weighted values, then one each.  A wait
    // names a completion by its parity, so none may run two completions ahead of a role that waits for it:
    //   sready(c), ofull(c), kvfull(c), kvempty(c)  two barriers in turn each: the states' chain and the
    //              outputs', or two state products, run up to a chunk apart;
    //   B_CLEAN    completes once, in a last chunk with rows past the prompt's end;
    //   all others are completed again only after what waits for them has passed.
    enum { B_SFULL, B_PREADY, B_KVFULL, B_KVEMPTY = B_KVFULL + 2, B_SREADY = B_KVEMPTY + 2, B_OFULL = B_SREADY + 2, B_OEMPTY = B_OFULL + 2, B_CLEAN, B_DRAIN };
    __device__ uint32_t kvfull(int c) const { return one(B_KVFULL + (c & 1)); }
    __device__ uint32_t kvempty(int c) const { return one(B_KVEMPTY + (c & 1)); }
    __device__ uint32_t sready(int c) const { return one(B_SREADY + (c & 1)); }
    __device__ uint32_t ofull(int c) const { return one(B_OFULL + (c & 1)); }
    __device__ uint32_t bar(int i) const { return ptx::smem_u32(bars + i); }
    __device__ uint32_t full(int s) const { return bar(s); }
    __device__ uint32_t empty(int s) const { return bar(Cf::NSLOT + s); }
    __device__ uint32_t vready(int s) const { return bar(2 * Cf::NSLOT + s); }
    __device__ uint32_t vfree(int s) const { return bar(2 * Cf::NSLOT + Cf::NVB + s); }
    __device__ uint32_t one(int i) const { return bar(2 * Cf::NSLOT + 2 * Cf::NVB + i); }
    __device__ uint8_t *slot(int t) const { return base + (t % Cf::NSLOT) * Cf::TILE; }
    __device__ uint8_t *vbuf(int i) const { return base + Cf::OFF_V + (i % Cf::NVB) * Cf::VITEM; }
    __device__ uint8_t *simg() const { return base + Cf::OFF_S; }
    // tile numbers of chunk c in landing order
    __device__ static int tv(int c) { return Cf::TPC * c; }
    __device__ static int tk(int c) { return Cf::TPC * c + 1; }
    __device__ static int tq(int c) { return Cf::TPC * c + 2; }
    // `count` of the RELEASE arrivals that free tile t's slot: SHARE by the warps that read it or saw the scores
    // made of it, 1 by those that see its last product complete
    __device__ void release(int t, int count) const { ptx::mbar_arrive_n(empty(t % Cf::NSLOT), count); }

    __device__ void init_barriers() const {
        for (int s = 0; s < Cf::NSLOT; ++s) {
            ptx::mbar_init(full(s), 1);          // producer (+ bytes)
            ptx::mbar_init(empty(s), Cf::RELEASE);
        }
        for (int s = 0; s < Cf::NVB; ++s) {
            ptx::mbar_init(vready(s), 4);
            ptx::mbar_init(vfree(s), 1);
        }
        ptx::mbar_init(one(B_SFULL), 1);
        ptx::mbar_init(one(B_PREADY), STATES ? 1 : Cf::XW);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(one(B_KVFULL + i), 1);
            ptx::mbar_init(one(B_KVEMPTY + i), Cf::UW);
            ptx::mbar_init(one(B_SREADY + i), Cf::UW);
            ptx::mbar_init(one(B_OFULL + i), 1);
        }
        ptx::mbar_init(one(B_OEMPTY), Cf::OW);
        ptx::mbar_init(one(B_CLEAN), Cf::TW);
        ptx::mbar_init(one(B_DRAIN), STATES ? 1 : 2);
    }
    // Waits for completion number `k` (from 0) of a barrier; false: gave up.  A role that gives up stops,
    // and those that wait for it give up in turn.
    __device__ bool wait(uint32_t br, int k, int code) const { return mbar_wait_patient(br, k & 1, a.wd, code); }
    __device__ int chunks() const { return (end - begin + Cf::C - 1) / Cf::C; }
    __device__ int tokens(int c) const { return min(Cf::C, end - begin - c * Cf::C); }

    // ------------------------------------------------------------ TMA producer (one thread)
    __device__ void producer(const DecayMaps &m) const {
        const uint64_t once = ptx::l2_evict_first();
        const int nc = chunks();
        int t = 0;
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            const int n = begin + c * Cf::C;
            for (int w = 0; w < Cf::TPC; ++w, ++t) {
                const int s = t % Cf::NSLOT;
                if (t >= Cf::NSLOT && !(ok = wait(empty(s), t / Cf::NSLOT - 1, WD_DC_EMPTY))) break;
                const bool isv = w == 0, isk = w == 1;
                const CUtensorMap *map = isk ? &m.k : isv ? &m.v : &m.q;
                const MapCoord mc = map_coord(n, h, isk ? m.swap_k : isv ? m.swap_v : m.swap_q);
                ptx::mbar_arrive_expect_tx(full(s), Cf::TILE);
#pragma unroll
                for (int at = 0; at < Cf::NAT; ++at)
                    ptx::tma_load_4d_hint(ptx::smem_u32(slot(t)) + at * Cf::SUB, map, full(s), at * Cf::AW, mc.y, mc.z, b,
                                          once);
            }
        }
        // no copy may be in flight when the CTA ends: the last tile of each slot has landed
        for (int u = max(0, t - Cf::NSLOT); u < t; ++u)
            ptx::mbar_wait_bounded(full(u % Cf::NSLOT), (u / Cf::NSLOT) & 1, a.wd, WD_DC_FULL, kWaitLimitNs);
    }

    // ------------------------------------------------------------ MMA issuers (one thread each)
    // An operand's descriptor: the address in 16-byte units in the low word, its layout in the high one.  The
    // thread that issues the products has few instructions to spare for each (a product of 128 x 128 x 16
    // takes 64 cycles), so steps along an operand are additions of constants to the low word.
    struct Operand {
        uint32_t lo, hi;
        __device__ Operand(uint32_t addr, uint32_t atom) {
            const uint64_t d = ptx::smem_desc(addr, atom, 8 * Cf::ROWB, Cf::LAYOUT);
            lo = static_cast<uint32_t>(d);
            hi = static_cast<uint32_t>(d >> 32);
        }
        __device__ Operand(uint32_t l, uint32_t h, int) : lo(l), hi(h) {}
        __device__ Operand operator+(uint32_t bytes) const { return Operand(lo + (bytes >> 4), hi, 0); }
        // the atoms behind the first one moved by `bytes`
        __device__ Operand right(uint32_t bytes) const { return Operand(lo + (bytes >> 4 << 16), hi, 0); }
    };
    __device__ static Operand kmajor(uint32_t addr) { return Operand(addr, 16); }
    __device__ static Operand mnmajor(uint32_t addr, uint32_t atom) { return Operand(addr, atom); }
    // 16 features along a K-major tile, 16 rows along an MN-major one: bytes
    static constexpr uint32_t kstep(int kk) { return (kk / (Cf::AW / 16)) * Cf::SUB + (kk % (Cf::AW / 16)) * 32; }
    static constexpr uint32_t rstep(int kk) { return kk * 16 * Cf::ROWB; }
    template <uint32_t ID, bool ACC>
    __device__ static void mma(uint32_t d, Operand x, Operand y) {
        ptx::mma_bf16_ss(d, x.lo, x.hi, y.lo, y.hi, ID, ACC);
    }
    // scores and outputs
    __device__ void mma_outputs() const {
        const int nc = chunks();
        for (int c = 0; c < nc; ++c) {
            if (!wait(full(tk(c) % Cf::NSLOT), tk(c) / Cf::NSLOT, WD_DC_FULL) ||
                !wait(full(tq(c) % Cf::NSLOT), tq(c) / Cf::NSLOT, WD_DC_FULL))
                break;
            // a chunk with rows past the prompt's end: once those are cleared
            if (tokens(c) < Cf::C && !wait(one(B_CLEAN), 0, WD_DC_VALUE)) break;
            const Operand qd = kmajor(ptx::smem_u32(slot(tq(c)))), kd = kmajor(ptx::smem_u32(slot(tk(c))));
            // The scores' columns were last read by the score warps (B_PREADY).  Where P lies in them, the product
            // with the values reads it there: that product has another shape and another accumulator, so that
            // its place in the order of issue does not keep it ahead of this one.
            if (!Cf::POWN && c > 0) {
                if (!wait(ofull(c - 1), (c - 1) >> 1, WD_DC_OUT)) break;
                ptx::tc_fence_after_sync();
            }
            constexpr uint32_t IDS = ptx::idesc_bf16_f32(128, 128, 0, 0), IDO = ptx::idesc_bf16_f32(128, D, 0, 1);
            mma<IDS, false>(tmem, qd, kd);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) mma<IDS, true>(tmem, qd + kstep(kk), kd + kstep(kk));
            ptx::mma_commit(one(B_SFULL));
            if (!wait(sready(c), c >> 1, WD_DC_STATE) || (c > 0 && !wait(one(B_OEMPTY), c - 1, WD_DC_OUT))) break;
            ptx::tc_fence_after_sync();
            const Operand sd = mnmajor(ptx::smem_u32(simg()), D * Cf::ROWB);
            mma<IDO, false>(tmem + Cf::T_OI, qd, sd + Cf::SIMG);
            mma<IDO, true>(tmem + Cf::T_OI, qd, sd);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) {
                mma<IDO, true>(tmem + Cf::T_OI, qd + kstep(kk), sd + (Cf::SIMG + rstep(kk)));
                mma<IDO, true>(tmem + Cf::T_OI, qd + kstep(kk), sd + rstep(kk));
            }
            if (!wait(full(tv(c) % Cf::NSLOT), tv(c) / Cf::NSLOT, WD_DC_FULL) || !wait(one(B_PREADY), c, WD_DC_SCORE)) break;
            ptx::tc_fence_after_sync();
            const Operand vd = mnmajor(ptx::smem_u32(slot(tv(c))), Cf::SUB);
#pragma unroll
            for (int kk = 0; kk < Cf::C / 16; ++kk) {
                const Operand v = vd + rstep(kk);
                ptx::mma_bf16_ts(tmem + Cf::T_OA, tmem + Cf::T_P + Cf::PSTEP * kk, v.lo, v.hi, IDO, kk > 0);
            }
            ptx::mma_commit(ofull(c));
        }
        drain();
    }
    // State product, item by item.  Products that add to the same columns must all have one shape: only then
    // does the order in which they were issued hold.  With KVN = 2 the low part therefore goes out as the
    // right half of a product as wide as that of the two others, with zeros for its left half.
    __device__ void mma_states() const {
        const int nc = chunks();
        const Operand v0 = mnmajor(ptx::smem_u32(vbuf(0)), Cf::VSUB);
        const uint32_t zeros = ptx::smem_u32(base + Cf::OFF_Z);
        const Operand low0 = mnmajor(zeros, ptx::smem_u32(vbuf(0)) + 2 * Cf::VPART - zeros);
        static_assert(Cf::NIT % Cf::NVB == 0, "an item's buffer is known at compile time");
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            if (!wait(full(tk(c) % Cf::NSLOT), tk(c) / Cf::NSLOT, WD_DC_FULL)) break;
            if (c >= Cf::KB && !wait(kvempty(c - Cf::KB), (c - Cf::KB) >> 1, WD_DC_STATE)) break;
            const uint32_t to = tmem + Cf::T_KV + c % Cf::KB * Cf::KVC;
            if (tokens(c) < Cf::C && !wait(one(B_CLEAN), 0, WD_DC_VALUE)) break;
            const Operand kd = mnmajor(ptx::smem_u32(slot(tk(c))), D == 128 ? Cf::SUB : 0);
#pragma unroll
            for (int it = 0; it < Cf::NIT; ++it) {
                constexpr int NB = Cf::NVB;
                if (!(ok = ok && wait(vready(it % NB), (c * Cf::NIT + it) / NB, WD_DC_VALUE))) break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < Cf::IT / 16; ++kk) {
                    const Operand k = kd + rstep(it * (Cf::IT / 16) + kk), v = v0 + (it % NB * Cf::VITEM + rstep(kk));
                    constexpr uint32_t ID = ptx::idesc_bf16_f32(Cf::KVM, Cf::KVN * D, 1, 1), ID1 = ptx::idesc_bf16_f32(Cf::KVM, D, 1, 1);
                    if constexpr (Cf::KVN == 1) {  // small parts first
                        if (it == 0 && kk == 0) mma<ID1, false>(to, k, v + 2 * Cf::VPART);
                        else mma<ID1, true>(to, k, v + 2 * Cf::VPART);
                        mma<ID1, true>(to, k, v + Cf::VPART);
                        mma<ID1, true>(to, k, v);
                    } else {
                        if (it == 0 && kk == 0) mma<ID, false>(to, k, v);
                        else mma<ID, true>(to, k, v);
                        if constexpr (Cf::KVN == 2) mma<ID, true>(to, k, low0.right(it % NB * Cf::VITEM + rstep(kk)));
                    }
                }
                ptx::mma_commit(vfree(it % NB));
            }
            if (!ok) break;
            ptx::mma_commit(kvfull(c));
        }
        drain();
    }
    // every MMA, and the arrivals of its commit, completes before TMEM is released
    __device__ void drain() const {
        ptx::mma_commit(one(B_DRAIN));
        wait(one(B_DRAIN), 0, WD_DC_DRAIN);
    }

    // ------------------------------------------------------------ score warps (row i per thread)
    // Columns go in groups of 16, which the XG warps of a row take in turn; a group's P is 16 bf16 in 8
    // columns.  The weights scale g^{i-j} of the diagonal block stay in registers
    // (0 right of the diagonal); left of it they are g^{i - 32 blk - 31} * scale g^{31 - (j - 32 blk)}, both
    // powers >= 0.
    __device__ void scores(int xw, int lane) const {
        constexpr int XG = Cf::XG == 2 ? 2 : 1, GS = 2 / XG;  // groups of a 32-column block that this warp takes
        const int w = xw & 3, x0 = xw >> 2;
        const uint32_t row = tmem + (static_cast<uint32_t>(32 * w) << 16), to = row + Cf::T_P;
        float dw[16 * GS];
#pragma unroll
        for (int m = 0; m < 16 * GS; ++m) dw[m] = 16 * x0 + m <= lane ? a.scale * pw[lane - m - 16 * x0] : 0.f;
        const int nc = chunks();
        for (int c = 0; c < nc; ++c) {
            if (!wait(one(B_SFULL), c, WD_DC_SCORE)) break;
            if (xw == 0 && lane == 0) release(tk(c), Cf::SHARE);  // multiplied by the queries
            ptx::tc_fence_after_sync();
#pragma unroll 1
            for (int g = x0; g < 2 * w; g += XG) {
                uint32_t s[16], p[8];
                ptx::tmem_ld(row + 16 * g, s);
                const float f = pw[32 * (w - (g >> 1) - 1) + 1 + lane];
                const float4 *l4 = reinterpret_cast<const float4 *>(lead + 16 * (g & 1));
                ptx::tmem_wait_ld();
                ptx::tmem_pin(s);
#pragma unroll
                for (int m = 0; m < 16; m += 4) {
                    const float4 l = l4[m / 4];
                    const float2 x = mul2(s[m], s[m + 1], mul2(f, f, l.x, l.y)), y = mul2(s[m + 2], s[m + 3], mul2(f, f, l.z, l.w));
                    p[m / 2] = pack_bf16x2(x.x, x.y);
                    p[m / 2 + 1] = pack_bf16x2(y.x, y.y);
                }
                ptx::tmem_st(to + Cf::PSTEP * g, p);
            }
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                uint32_t s[16], p[8];
                const int gd = 2 * w + x0 + g;
                ptx::tmem_ld(row + 16 * gd, s);
                ptx::tmem_wait_ld();
                ptx::tmem_pin(s);
#pragma unroll
                for (int m = 0; m < 16; m += 2) {
                    const float2 x = mul2(s[m], s[m + 1], make_float2(dw[16 * g + m], dw[16 * g + m + 1]));
                    p[m / 2] = pack_bf16x2(x.x, x.y);
                }
                ptx::tmem_st(to + Cf::PSTEP * gd, p);
            }
            const uint32_t zero[8] = {};
#pragma unroll 1
            for (int g = 2 * w + 2 + x0; g < 8; g += XG) ptx::tmem_st(to + Cf::PSTEP * g, zero);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            warp_arrive(one(B_PREADY), lane);
        }
    }
    __device__ static float2 mul2(float x, float y, float u, float v) { return mul2(__float_as_uint(x), __float_as_uint(y), make_float2(u, v)); }
    // two products in one instruction
    __device__ static float2 mul2(uint32_t x, uint32_t y, float2 b) {
        float2 r;
        asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n}\n"
            : "=f"(r.x), "=f"(r.y)
            : "r"(x), "r"(y), "f"(b.x), "f"(b.y));
        return r;
    }

    // ------------------------------------------------------------ value warps
    // Thread: one token row of an item, a share of its 16-byte pieces.  The TG warpgroups take the items in
    // turn.
    __device__ void values(int tid, int lane) const {
        constexpr int PARTS = 128 / Cf::IT, PCS = D / 8 / PARTS;
        static_assert(PCS >= 1, "a thread has a piece to write");
        const int tg = tid >> 7;
        tid &= 127;
        const int r = tid % Cf::IT, part = tid / Cf::IT;
        const int nc = chunks();
        for (int c = 0; c < nc; ++c) {
            const int n = tokens(c);
            if (!wait(full(tv(c) % Cf::NSLOT), tv(c) / Cf::NSLOT, WD_DC_FULL)) return;
            uint8_t *v = slot(tv(c));
            if (n < Cf::C) {
                // rows past the end multiply zeros: what lies there may be NaN
                if (!wait(full(tk(c) % Cf::NSLOT), tk(c) / Cf::NSLOT, WD_DC_FULL)) return;
                if (tid >= n)
                    for (int j = 0; j < Cf::NAT * ROWP; ++j) {
                        const uint32_t off = (j / ROWP) * Cf::SUB + swz_chunk<Cf::AW>(tid, j % ROWP);
                        if (tg == 0) *reinterpret_cast<uint4 *>(v + off) = make_uint4(0, 0, 0, 0);
                        if (tg == Cf::TG - 1) *reinterpret_cast<uint4 *>(slot(tk(c)) + off) = make_uint4(0, 0, 0, 0);
                    }
                ptx::fence_proxy_async_smem();
                warp_arrive(one(B_CLEAN), lane);
            }
#pragma unroll 1
            for (int it = tg; it < Cf::NIT; it += Cf::TG) {
                const int i = c * Cf::NIT + it, tok = it * Cf::IT + r;
                if (i >= Cf::NVB && !wait(vfree(i % Cf::NVB), i / Cf::NVB - 1, WD_DC_VALUE)) return;
                uint8_t *dst = vbuf(i);
                const bool live = tok < n;
                const float w = live ? pw[n - 1 - tok] : 0.f;
#pragma unroll 2
                for (int j = 0; j < PCS; ++j) {
                    const int pc = part * PCS + j, at = pc / ROWP, cc = pc % ROWP;
                    uint4 hi = make_uint4(0, 0, 0, 0), mid = hi, lo = hi;
                    if (live) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(v + at * Cf::SUB + swz_chunk<Cf::AW>(tok, cc));
                        split(x.x, w, hi.x, mid.x, lo.x);
                        split(x.y, w, hi.y, mid.y, lo.y);
                        split(x.z, w, hi.z, mid.z, lo.z);
                        split(x.w, w, hi.w, mid.w, lo.w);
                    }
                    uint8_t *d = dst + at * Cf::VSUB + swz_chunk<Cf::AW>(r, cc);
                    *reinterpret_cast<uint4 *>(d) = hi;
                    *reinterpret_cast<uint4 *>(d + Cf::VPART) = mid;
                    *reinterpret_cast<uint4 *>(d + 2 * Cf::VPART) = lo;
                }
                ptx::fence_proxy_async_smem();  // written for the MMA; V read before its slot is filled again
                warp_arrive(vready(i % Cf::NVB), lane);
            }
            if (lane == 0) release(tv(c), Cf::SHARE / Cf::TW + (STATES && tid == 0 && tg == 0 ? 1 : 0));
        }
    }
    static constexpr int ROWP = Cf::ROWB / 16;  // 16-byte pieces of a row of one atom
    // w times a pair of values, as three bf16 parts that add up to the fp32 products: the upper 16 bits, the
    // upper 16 bits of what is left (exact differences), and the rest, at most 8 significant bits
    __device__ static void split(uint32_t x, float w, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
        float2 v = mul2(x << 16, x & 0xFFFF0000u, make_float2(w, w));
        hi = upper(v);
        v = less(v, hi);
        mid = upper(v);
        lo = upper(less(v, mid));
    }
    __device__ static uint32_t upper(float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); }
    // v minus a pair of bf16, by multiply-adds that take them as they are
    __device__ static float2 less(float2 v, uint32_t h) {
        float2 r;
        asm("{\n\t.reg .b16 x, y, m;\n\tmov.b32 {x, y}, %4;\n\tmov.b16 m, 0xBF80;\n\t"
            "fma.rn.f32.bf16 %0, x, m, %2;\n\tfma.rn.f32.bf16 %1, y, m, %3;\n\t}\n"
            : "=f"(r.x), "=f"(r.y)
            : "f"(v.x), "f"(v.y), "r"(h));
        return r;
    }
    // two multiply-adds in one instruction
    __device__ static float2 fma2(float2 x, float2 y, float2 z) {
        float2 r;
        asm("{\n\t.reg .b64 p, q, s;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 s, {%6, %7};\n\t"
            "fma.rn.f32x2 p, p, q, s;\n\tmov.b64 {%0, %1}, p;\n}\n"
            : "=f"(r.x), "=f"(r.y)
            : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
        return r;
    }
    __device__ static float2 pair(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }

    // ------------------------------------------------------------ state warps
    // Elements of the state a thread holds.  d = 128: row f = 32 sub + lane, 64 columns from col0.  Else the
    // 16-lane fragments of an M = 64 product: pairs of neighbouring columns, pair p in row f + 8 (p & 1) and
    // column col0 + 8 (p >> 1) + 2 (lane & 3).
    struct Piece {
        uint32_t row;  // TMEM lanes of this warp
        int f, col0;
        __device__ Piece(uint32_t tmem, int uw, int lane) {
            const int sub = uw & 3;
            row = tmem + (static_cast<uint32_t>(32 * sub) << 16);
            if constexpr (D == 128) {
                f = 32 * sub + lane;
                col0 = 64 * (uw >> 2);
            } else {
                f = (16 * sub + (lane >> 2)) % D;
                col0 = (16 * sub / D) * 16;
            }
        }
        static constexpr int RUN = D == 128 ? 4 : 2;  // elements of one access to a row in memory
        __device__ int offset(int i, int lane) const {
            if constexpr (D == 128) return f * D + col0 + RUN * i;
            else return (f + 8 * (i & 1)) * D + col0 + 8 * (i >> 1) + 2 * (lane & 3);
        }
    };
    using Run = typename std::conditional<D == 128, float4, float2>::type;

    __device__ void load_state(float (&st)[Cf::NCOL], const Piece &pc, int lane) const {
        auto add = [&](const float *src, float w) {
#pragma unroll
            for (int i = 0; i < Cf::NCOL / Piece::RUN; ++i) {
                const Run x = *reinterpret_cast<const Run *>(src + pc.offset(i, lane));
                const float *e = &x.x;
#pragma unroll
                for (int u = 0; u < Piece::RUN; ++u) st[Piece::RUN * i + u] = fmaf(w, e[u], st[Piece::RUN * i + u]);
            }
        };
#pragma unroll
        for (int i = 0; i < Cf::NCOL; ++i) st[i] = 0.f;
        if (a.nseg > 1)
            for (int p = 0; p * a.piece <= begin; ++p) add(wsp + (size_t)p * D * D, decay_pow(lg, (float)(begin - p * a.piece)));
        else if (pool) add(pool, 1.f);
    }
    __device__ static void store_state(const float (&st)[Cf::NCOL], float *dst, const Piece &pc, int lane) {
#pragma unroll
        for (int i = 0; i < Cf::NCOL / Piece::RUN; ++i) {
            Run x;
            float *e = &x.x;
#pragma unroll
            for (int u = 0; u < Piece::RUN; ++u) e[u] = st[Piece::RUN * i + u];
            *reinterpret_cast<Run *>(dst + pc.offset(i, lane)) = x;
        }
    }
    // this thread's part of the state as two bf16 operand images, the rounded state and the rounded rest
    __device__ static void put_state(const float (&st)[Cf::NCOL], uint8_t *img, const Piece &pc, int lane) {
        auto low = [](float x, float y, uint32_t hi) {
            const float2 r = less(make_float2(x, y), hi);
            return pack_bf16x2(r.x, r.y);
        };
        if constexpr (D == 128) {
#pragma unroll
            for (int j = 0; j < Cf::NCOL / 8; ++j) {
                const int q = pc.col0 / 8 + j;
                uint8_t *to = img + (q / ROWP) * D * Cf::ROWB + swz_chunk<Cf::AW>(pc.f, q % ROWP);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = st[8 * j + 2 * i], y = st[8 * j + 2 * i + 1];
                    hi[i] = pack_bf16x2(x, y);
                    lo[i] = low(x, y, hi[i]);
                }
                *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(to + Cf::SIMG) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        } else {
            // pairs 4q .. 4q + 3 are four 8 x 8 blocks: rows f and f + 8 of two neighbouring 16-byte pieces
            const int blk = lane >> 3;
            const int row = pc.f - (lane >> 2) + 8 * (blk & 1) + (lane & 7);
#pragma unroll
            for (int q = 0; q < Cf::NCOL / 8; ++q) {
                const uint32_t to = ptx::smem_u32(img + swz_chunk<Cf::AW>(row, pc.col0 / 8 + 2 * q + (blk >> 1)));
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = st[8 * q + 2 * i], y = st[8 * q + 2 * i + 1];
                    hi[i] = pack_bf16x2(x, y);
                    lo[i] = low(x, y, hi[i]);
                }
                ptx::stmatrix_x4(to, hi);
                ptx::stmatrix_x4(to + Cf::SIMG, lo);
            }
        }
        ptx::fence_proxy_async_smem();
    }
    // S <- g S + this chunk's product
    __device__ void add_product(float (&st)[Cf::NCOL], const DecaySplit &g, const Piece &pc, int c) const {
#pragma unroll
        for (int i0 = 0; i0 < Cf::NCOL; i0 += 8) {
            uint32_t x[Cf::KVN][8];
            const int col = D == 128 ? i0 : 2 * i0;  // 8 columns of a row, or 16 columns of two half rows
#pragma unroll
            for (int p = 0; p < Cf::KVN; ++p) {
                const uint32_t at = pc.row + Cf::T_KV + c % Cf::KB * Cf::KVC + p * D + pc.col0 + col;
                if constexpr (D == 128) ptx::tmem_ld(at, x[p]);
                else ptx::tmem_ld_16x256(at, x[p]);
            }
            ptx::tmem_wait_ld();
#pragma unroll
            for (int p = 0; p < Cf::KVN; ++p) ptx::tmem_pin(x[p]);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 t = pair(x[Cf::KVN - 1][i], x[Cf::KVN - 1][i + 1]);
#pragma unroll
                for (int p = Cf::KVN - 2; p >= 0; --p) t = fma2(pair(x[p][i], x[p][i + 1]), make_float2(1.f, 1.f), t);
                const float2 v = make_float2(st[i0 + i], st[i0 + i + 1]);
                t = fma2(v, make_float2(g.hi, g.hi), fma2(v, make_float2(g.lo, g.lo), t));
                st[i0 + i] = t.x;
                st[i0 + i + 1] = t.y;
            }
        }
    }
    __device__ void states(const DecayMaps &m, int uw, int lane) const {
        const Piece pc(tmem, uw, lane);
        float st[Cf::NCOL];
        if constexpr (STATES) {
#pragma unroll
            for (int i = 0; i < Cf::NCOL; ++i) st[i] = 0.f;
        } else {
            load_state(st, pc, lane);
            put_state(st, simg(), pc, lane);
            warp_arrive(sready(0), lane);
        }
        const DecaySplit whole(lg, (float)Cf::C);
        const int nc = chunks();
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            const int n = tokens(c);
            if (!(ok = wait(kvfull(c), c >> 1, WD_DC_STATE))) break;
            if (uw == 0 && lane == 0) release(tk(c), STATES ? Cf::RELEASE : 1);
            ptx::tc_fence_after_sync();
            DecaySplit g = whole;
            if (n < Cf::C) g = DecaySplit(lg, (float)n);
            add_product(st, g, pc, c);
            ptx::tc_fence_before_sync();
            warp_arrive(kvempty(c), lane);
            if constexpr (!STATES) {
                if (c + 1 < nc) {
                    // the next chunk's images go where this one's are, once those have been multiplied
                    if (!(ok = wait(ofull(c), c >> 1, WD_DC_OUT))) break;
                    put_state(st, simg(), pc, lane);
                    warp_arrive(sready(c + 1), lane);
                }
                if (!Cf::ZW) ok = output_chunk(m, c, uw, lane);
            }
        }
        if constexpr (STATES) {
            store_state(st, wsp + (size_t)(seg + 1) * D * D, pc, lane);
        } else {
            if (ok && pool && end == decay_len(a, b)) store_state(st, pool, pc, lane);
            if (!Cf::ZW && lane == 0) ptx::bulk_wait_group_read<0>();
        }
    }

    // ------------------------------------------------------------ output warps (row i per thread)
    __device__ void outputs(const DecayMaps &m, int zw, int lane) const {
        const int nc = chunks();
        for (int c = 0; c < nc; ++c)
            if (!output_chunk(m, c, zw, lane)) break;
        if (lane == 0) ptx::bulk_wait_group_read<0>();  // staged rows have left before the CTA's memory goes
    }
    __device__ bool output_chunk(const DecayMaps &m, int c, int sub, int lane) const {
        const int r = 32 * sub + lane, n = tokens(c);
        const float go = a.scale * pw[r + 1];
        const uint32_t row = tmem + (static_cast<uint32_t>(32 * sub) << 16);
        if (lane == 0 && c > 0) {  // the staged rows of the last chunk have left
            ptx::bulk_wait_group_read<0>();
            if (D == 128) release(tq(c - 1), Cf::SHARE / Cf::OW);
        }
        __syncwarp();
        if (!wait(ofull(c), c >> 1, WD_DC_OUT)) return false;
        if (sub == 0 && lane == 0) {  // the chunk's products are done
            release(tv(c), 1);
            release(tq(c), D == 128 ? 1 : Cf::RELEASE);  // d = 128: and by the warps whose rows leave from it
        }
        ptx::tc_fence_after_sync();
        uint8_t *stg = (D == 128 ? slot(tq(c)) : base + Cf::OFF_O) + 32 * sub * Cf::ROWB;
#pragma unroll 1
        for (int j = 0; j < D / 8; j += 2) {
            uint32_t x[16], y[16], o[8];
            ptx::tmem_ld(row + Cf::T_OA + 8 * j, x);
            ptx::tmem_ld(row + Cf::T_OI + 8 * j, y);
            ptx::tmem_wait_ld();
            ptx::tmem_pin(x);
            ptx::tmem_pin(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = fma2(make_float2(go, go), pair(y[2 * i], y[2 * i + 1]), pair(x[2 * i], x[2 * i + 1]));
                o[i] = pack_bf16x2(v.x, v.y);
            }
            if (r >= n)  // rows past the prompt's end are zeros
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = 0u;
            uint8_t *dst = stg + (j / ROWP) * Cf::SUB;
            *reinterpret_cast<uint4 *>(dst + swz_chunk<Cf::AW>(lane, j % ROWP)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + swz_chunk<Cf::AW>(lane, j % ROWP + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        ptx::tc_fence_before_sync();
        ptx::fence_proxy_async_smem();
        warp_arrive(one(B_OEMPTY), lane);
        if (lane == 0) {
            const int n0 = begin + c * Cf::C + 32 * sub;
            const MapCoord mc = map_coord(n0, h, m.swap_o);
            if (n0 < a.N)
#pragma unroll
                for (int at = 0; at < Cf::NAT; ++at)
                    ptx::tma_store_4d_hint(&m.o, ptx::smem_u32(stg + at * Cf::SUB), at * Cf::AW, mc.y, mc.z, b,
                                           ptx::l2_evict_first());
            ptx::bulk_commit_group();
        }
        return true;
    }
};

// Changes the registers a thread of this warpgroup may use from FROM to TO (0: no split).
template <int FROM, int TO>
__device__ __forceinline__ void regs() {
    if constexpr (FROM > 0 && TO > 0 && TO < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TO));
    if constexpr (FROM > 0 && TO > 0 && TO > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TO));
}

template <int D, bool STATES>
__global__ void __launch_bounds__(DecayTc<D, STATES>::THREADS, D == 32 ? 2 : 1)
    decay_tc_kernel(const __grid_constant__ DecayMaps m, const __grid_constant__ DecayArgs a) {
    using Cf = DecayTc<D, STATES>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = align1024(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = STATES ? a.npiece : a.nseg, span = STATES ? a.piece : a.seg;
    const int run = blockIdx.x / per, seg = blockIdx.x - run * per;
    const int at = run / a.H, h = run - at * a.H, b = STATES ? at : decay_row(a, at, base), bh = STATES ? run : b * a.H + h;
    const int slot = decay_slot(a, b);
    const int L = slot < 0 ? 0 : decay_len(a, b);
    const int begin = seg * span, stop = min(begin + span, a.N);
    float *pool = a.S && slot >= 0 ? a.S + ((size_t)slot * a.H + h) * D * D : nullptr;
    float *wsp = a.ws + (size_t)bh * (1 + a.npiece) * D * D;
    if (STATES && seg == 0)  // the second launch may overwrite the pool while others still read the entering state
        for (int i = tid; i < D * D / 4; i += Cf::THREADS)
            reinterpret_cast<float4 *>(wsp)[i] =
                pool ? reinterpret_cast<const float4 *>(pool)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    const int end = min(stop, L);
    if (end > begin) {
        const float lg = decay_log(a.log_decay, h);
        uint64_t *bars = reinterpret_cast<uint64_t *>(base + Cf::OFF_CTRL);
        uint32_t *tslot = reinterpret_cast<uint32_t *>(base + Cf::OFF_CTRL + 508);
        float *pw = reinterpret_cast<float *>(base + Cf::OFF_PW);
        DecayUnit<D, STATES> u{a, base, bars, pw, pw + 132, 0u, b, h, begin, end, lg, pool, wsp, seg};
        if (tid == 0) {
            u.init_barriers();
            ptx::fence_mbar_init();
        }
        if (tid < Cf::ZTILE / 16) reinterpret_cast<uint4 *>(base + Cf::OFF_Z)[tid] = make_uint4(0, 0, 0, 0);
        // decay_row's scratch lies where the first tile lands; the zeros are read by products
        if (a.sorted || Cf::ZTILE) ptx::fence_proxy_async_smem();
        if (tid < 129) pw[tid] = decay_pow(lg, (float)tid);
        else if (tid < 161) pw[132 + tid - 129] = a.scale * decay_pow(lg, (float)(31 - (tid - 129)));
        if (warp == 0) {
            ptx::tmem_alloc(ptx::smem_u32(tslot), Cf::TCOLS);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
        u.tmem = *tslot;
        constexpr int X = Cf::XW, T = X + Cf::TW, U = T + Cf::UW, Z = U + Cf::ZW, RL = Cf::RL;
        if (warp < X) {
            regs<RL, Cf::RX>();
            if constexpr (!STATES) u.scores(warp, lane);
            regs<Cf::RX, RL>();  // the code behind the roles is common to all
        } else if (warp < T) {
            regs<RL, Cf::RT>();
            u.values(tid - 32 * X, lane);
            regs<Cf::RT, RL>();
        } else if (warp < U) {
            regs<RL, Cf::RU>();
            u.states(m, warp - T, lane);
            regs<Cf::RU, RL>();
        } else if (warp < Z) {
            regs<RL, Cf::RZ>();
            if constexpr (Cf::ZW > 0) u.outputs(m, warp - U, lane);
            regs<Cf::RZ, RL>();
        } else {
            regs<RL, Cf::RC>();
            if (lane == 0) {
                if (warp == Z) u.producer(m);
                else if (warp == Z + 1) u.mma_states();
                else if (!STATES && warp == Z + 2) u.mma_outputs();
            }
            __syncwarp();
            regs<Cf::RC, RL>();
        }
        ptx::tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            ptx::tc_fence_after_sync();
            ptx::tmem_dealloc(u.tmem, Cf::TCOLS);
        }
    } else if (STATES) {
        float4 *dst = reinterpret_cast<float4 *>(wsp + (size_t)(seg + 1) * D * D);
        for (int i = tid; i < D * D / 4; i += Cf::THREADS) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (!STATES) {
        // rows behind the last chunk (whose own rows past the end went out as zeros)
        const int z0 = max(begin, begin + (max(end - begin, 0) + Cf::C - 1) / Cf::C * Cf::C);
        __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.o) + b * a.lo.batch + h * a.lo.head;
        for (long long i = tid; i < (long long)(stop - z0) * (D / 8); i += Cf::THREADS)
            *reinterpret_cast<uint4 *>(op + (z0 + i / (D / 8)) * a.lo.tok + i % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace blin

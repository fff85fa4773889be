// k_mix_tc.cu -- the causal mix of linattn.cuh on the sm_100a tensor cores
// (bf16 rows, widths up to 128): the linear-attention forward, and each of
// the three products of its backward.
//
// The chunked form, chunks of 64 tokens.  With M the state entering a chunk
// (fp32, da x 64 of the dc columns), L its tokens, i and j places in it:
//   D1 = A B^T              scores                     M=64  N=64 K=da
//   P_ji = scale_p g^|j-i| D1_ji  (i <= j; walking backwards i >= j), bf16
//   D2 = P C                own chunk's answer         M=64  N=64 K=64
//   D3 = A M                the past's answer          M=64  N=64 K=da
//   D4 = B^T Cw             own chunk's state          M=128 N=3x64 K=64
//   y_j = D2_j + scale_i g^(j+1) D3_j                  (backwards g^(L-1-j))
//   M  <- M g^L + D4 (as in decay_of),  Cw_i = scale_w g^(L-1-i) c_i   (backwards g^(i+1))
// The decay is a constant of the lane, so every weight is a table of the 65
// powers g^0 .. g^64: the 64 x 64 mask lives in the score warps' registers.
//
// Roundings: A, B, C enter as they are.  P and the copy of M that D3 reads
// are rounded to bf16, one rounding for each term of y, as y itself has.  The
// state is carried in fp32 and is an output in fp32, so Cw goes in as three
// bf16 pieces, hi + mid + lo = w c exactly, side by side in D4's columns.
//
// One CTA owns one lane, one tile of 64 columns of c and one segment of the
// time axis, and walks its chunks.  24 warps: 0 TMA, 1-3 UMMA issue (D1; D4; D3
// and D2), 4-7 Cw, 8-11 scores, 12-19 state, 20-23 outputs.  Three issuing
// warps, not one: a section of waits, fence, issue and commit takes a warp 400
// to 700 cycles, four of them in a row more than anything else in a chunk.  The
// hand-overs are buffered in TMEM or shared memory, so the roles work on
// different chunks; the chain from chunk to chunk is only the state's update.
// A split time axis takes two passes: B and C alone for every segment's own
// state, the combine of linattn.cuh, then all segments at once.
//
// Measured: 8 x 2048 tokens, 16 heads of 128 x 64, 43 to 45 us with the clock for
// 206 MB (69 % of the copy rate), on 128 of the 148 SMs; the backward's dq and dk
// 128 to 141 us, dv 42 to 46.  No unit is at its limit there: of an SM's active
// cycles (about 2300 a chunk) the issue slots are busy for 57 %, tensor memory for
// 50, the tensor pipe for 44, the LSU's data pipe for 42; DRAM is at 49 %.  What is
// left are the hand-overs between the roles, each a chain of waits, fences and
// latencies: 1.2 of a scheduler's 6 warps are ready at a time.  (768 threads leave
// 80 registers a thread; the wide variant spills 12 bytes.)  One persistent CTA to
// an SM instead of one to a lane was slower at long sequences (220 us for the
// backward, 195 here) and faster at hundreds of single chunks (512 x 64 tokens: 288
// us, 338 here).
//
// The problems of a call (three in the backward) share one launch.  Every
// wait is bounded: past ~1 s the kernel records the site, stops issuing work,
// drains what it has in flight and returns.
#include <atomic>
#include <initializer_list>

#include "linattn.cuh"
#include "tc_ptx.cuh"

namespace m3 {
namespace mixtc {
using namespace ptx;

constexpr int Q = 64, DC = 64, DA = 128;               // chunk, columns of a tile, widest a, b and c rows
constexpr int W_TMA = 0, W_S = 1, W_D = 2, W_Y23 = 3, W_CW = 4, W_SC = 8, W_ST = 12, W_Y = 20, NWARPS = 24;
constexpr int THREADS = NWARPS * 32;

// ---- shared memory (bytes from a 1024-aligned base), all tiles 128B-swizzled.
// KD, the width that a and b rows are padded to (64 or 128): with 64 the
// tensor cores read and the state warps keep half, and more stages fit.
constexpr int SZ_T = Q * DC * 2, SZ_C = SZ_T;           // one 64 x 64 bf16 tile
template <int KD>
struct Lay {
    static constexpr int NST = KD == 64 ? 5 : 3;        // stages of A, B, C
    static constexpr int SZ_AB = Q * KD * 2, SZ_STAGE = 2 * SZ_AB + SZ_C;
    static constexpr int SZ_M = KD * DC * 2;
    static constexpr int OFF_STAGE = 0;
    static constexpr int OFF_CW = OFF_STAGE + NST * SZ_STAGE;   // 2 x 3 pieces
    static constexpr int OFF_P = OFF_CW + 2 * 3 * SZ_T;         // 2
    static constexpr int OFF_M = OFF_P + 2 * SZ_T;              // 2
    static constexpr int OFF_Y = OFF_M + 2 * SZ_M;              // 1
    static constexpr int OFF_PW = OFF_Y + SZ_T;                 // fp32 g^0 .. g^64, then g^n - 1
    static constexpr int OFF_BAR = OFF_PW + 2 * 72 * 4;
    static constexpr int OFF_MISC = OFF_BAR + 40 * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};
constexpr int NPW = 72, MAXST = 5;
constexpr int PFD = 3;                                  // chunks that the L2 prefetch runs ahead of the loads
enum {
    B_FULL = 0,                    // NST: a stage has arrived
    B_EMPTY = B_FULL + MAXST,      // NST: its readers are done
    // 2 of each from here on.  "Full" of an accumulator also says that the
    // operands it was made from may be overwritten: P and M (Y)
    B_CWFULL = B_EMPTY + MAXST,      // Cw in shared memory
    B_CWEMPTY = B_CWFULL + 2,
    B_PFULL = B_CWEMPTY + 2,       // masked scores in shared memory
    B_MFULL = B_PFULL + 2,         // the entering state in shared memory
    B_YFULL = B_MFULL + 2,         // both parts of the answer in TMEM
    B_YEMPTY = B_YFULL + 2,
    B_SFULL = B_YEMPTY + 2,        // 1 of each from here on.  Scores in TMEM
    B_SEMPTY,
    B_DFULL,                       // a chunk's own state in TMEM
    B_DEMPTY,
    B_ZERO,                        // rows behind the sequence are zeroed in B and C
    B_DRAIN = B_ZERO + 1,          // 3: every UMMA of an issuing warp is done
    NBAR = B_DRAIN + 3
};
static_assert(NBAR <= 40, "barriers");

constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_D = 64, COL_Y2 = 256, COL_Y3 = 384;   // 64, 3 x 64, 2 x 64, 2 x 64

constexpr int MAXP = 3;
struct Batch {
    CUtensorMap ma[MAXP], mb[MAXP], mc[MAXP], my[MAXP];
    MixArgs g[MAXP];
    unsigned first[MAXP + 1];      // first block of each problem
    int n;
    int *err;
};

// the upper half of an fp32 pattern (its first 8 significant bits), and of two
__device__ __forceinline__ float cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }
__device__ __forceinline__ uint32_t cut2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
// rounded to bf16, as one register
__device__ __forceinline__ uint32_t round2(f32x2 v) {
    float a, b;
    unpair(v, a, b);
    return pack_bf16(a, b);
}

template <bool SO, int KD>
__global__ void __launch_bounds__(THREADS, 1) k_mix_tc(const __grid_constant__ Batch P) {
    using L_ = Lay<KD>;
    constexpr int NST = L_::NST, SZ_AB = L_::SZ_AB, SZ_STAGE = L_::SZ_STAGE, SZ_M = L_::SZ_M;
    constexpr int OFF_STAGE = L_::OFF_STAGE, OFF_CW = L_::OFF_CW, OFF_P = L_::OFF_P, OFF_M = L_::OFF_M;
    constexpr int OFF_Y = L_::OFF_Y, OFF_PW = L_::OFF_PW, OFF_BAR = L_::OFF_BAR, OFF_MISC = L_::OFF_MISC;
    constexpr int NX = KD / 64;                         // 64-column halves of an A or B tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, l32 = tid & 31;
    int pi = 0;
    while (pi + 1 < P.n && blockIdx.x >= P.first[pi + 1]) pi++;
    const MixArgs &g = P.g[pi];
    const unsigned bid = blockIdx.x - P.first[pi];
    const unsigned ntile = (g.dc + DC - 1) / DC, nsb = SO ? g.nseg - 1 : g.nseg, H = (unsigned)g.H;
    const int seg = (int)(bid / ntile % nsb), p0 = (int)(bid % ntile) * DC;
    const unsigned lane32 = bid / ntile / nsb, b32 = lane32 / H, h32 = lane32 % H;
    const int64_t lane = lane32, b = b32, h = h32;
    const int64_t t_beg = seg_begin(seg, g.nseg, g.seg_len, g.reverse);
    const int ntok = (int)seg_tokens(seg, g.nseg, g.seg_len, g.reverse, lane_length(g.lengths, b, g.T));
    const int nch = (ntok + Q - 1) / Q;
    const bool rev = g.reverse != 0;
    auto bar = [&](int i) { return sbase + OFF_BAR + 8 * i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + OFF_MISC + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + OFF_MISC);
    float *pw = reinterpret_cast<float *>(sm + OFF_PW), *pm1 = pw + NPW;
    // chunk c of the walk starts at token chunk_t(c) of the segment and has chunk_n(c) tokens
    auto chunk_t = [&](int c) { return (rev ? nch - 1 - c : c) * Q; };
    auto chunk_n = [&](int c) { return min(Q, ntok - chunk_t(c)); };

    // a chunk's loads, by one lane
    const int ha = (int)(h32 / (unsigned)g.ra), hb = (int)(h32 / (unsigned)g.rb), hc = (int)(h32 / (unsigned)g.rc);
    auto load = [&](int c, int st) {
        const int t = (int)t_beg + chunk_t(c);
        const uint32_t s0 = sbase + OFF_STAGE + st * SZ_STAGE, fb = bar(B_FULL + st);
        mbar_expect_tx(fb, SO ? SZ_AB + SZ_C : SZ_STAGE);
#pragma unroll
        for (int x = 0; x < NX; x++) {
            if (!SO) tma_load4(s0 + x * SZ_T, &P.ma[pi], 64 * x, ha, t, (int)b32, fb);
            tma_load4(s0 + SZ_AB + x * SZ_T, &P.mb[pi], 64 * x, hb, t, (int)b32, fb);
        }
        tma_load4(s0 + 2 * SZ_AB, &P.mc[pi], p0, hc, t, (int)b32, fb);
    };

    // The first loads go out before anything else: the rest of the set-up
    // (about 3000 cycles) passes while they are on their way.
    if (tid == 0) {
        for (int i = 0; i < NST; i++) mbar_init(bar(B_FULL + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int c = 0; c < NST && c < nch; c++) load(c, c);
        for (int i = 0; i < NST; i++) mbar_init(bar(B_EMPTY + i), SO ? 5 : 6);   // D4, D2 and D3; four Cw warps
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(B_CWFULL + i), 4);
            mbar_init(bar(B_CWEMPTY + i), 1);
            mbar_init(bar(B_PFULL + i), 4);
            mbar_init(bar(B_MFULL + i), 8);
            mbar_init(bar(B_YFULL + i), 1);
            mbar_init(bar(B_YEMPTY + i), 4);
        }
        mbar_init(bar(B_SFULL), 1);
        mbar_init(bar(B_SEMPTY), 4);
        mbar_init(bar(B_DFULL), 1);
        mbar_init(bar(B_DEMPTY), 8);
        mbar_init(bar(B_ZERO), 4);
        for (int i = 0; i < 3; i++) mbar_init(bar(B_DRAIN + i), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_S) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid >= 128 && tid <= 128 + Q) decay_pow_f32(g.log_decay[h], tid - 128, pw[tid - 128], pm1[tid - 128]);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](int i, uint32_t parity, int site) { return warp_wait(bar(i), parity & 1, abort_flag, P.err, site); };
    auto arrive = [&](int i) {                          // once for a converged warp
        __syncwarp();
        if (l32 == 0) mbar_arrive(bar(i));
    };

    if (warp == W_TMA) {
        auto prefetch = [&](int c) {                    // a chunk on its way to L2
            const int t = (int)t_beg + chunk_t(c);
            for (int x = 0; x < g.da; x += 64) {
                if (!SO) tma_prefetch4(&P.ma[pi], x, ha, t, (int)b32);
                tma_prefetch4(&P.mb[pi], x, hb, t, (int)b32);
            }
            tma_prefetch4(&P.mc[pi], p0, hc, t, (int)b32);
        };
        if (elect_one())
            for (int c = NST; c < NST + PFD && c < nch; c++) prefetch(c);
        __syncwarp();
        int st = 0, k = 1;                              // stage, turn of the ring
        for (int c = NST; c < nch; c++) {
            if (!wait(B_EMPTY + st, k - 1, 101)) break;
            if (elect_one()) {
                load(c, st);
                if (c + PFD < nch) prefetch(c + PFD);
            }
            __syncwarp();
            if (++st == NST) st = 0, k++;
        }
        // every load issued lands before the CTA's memory goes away: the other
        // roles have waited for each stage, unless they gave up
        if (*abort_flag) {
            const long long t0 = clock64();
            for (int c = (nch > NST ? nch - NST : 0); c < nch; c++)
                while (!mbar_try(bar(B_FULL + c % NST), (c / NST) & 1) && clock64() - t0 < WAIT_LIMIT_CYCLES / 16) {
                }
        }
    } else if (warp < W_CW) {
        constexpr uint32_t id_kk = idesc(64, 64, 0, 0), id_kmn = idesc(64, 64, 0, 1), id_st = idesc(KD, 192, 1, 1);
        // Descriptor steps (16-byte units): a K-step of 16 is 32 bytes of a
        // K-major row (the second 64 columns lie half a tile further), and two
        // groups of 8 rows (MN) of an MN-major one.  The issue loops are
        // unrolled by four: rolled, the descriptor arithmetic between two
        // UMMAs takes 65 to 100 cycles, twice what a UMMA does (measured
        // beside busy warps: 3264 against 1437 cycles for a chunk's); unrolled
        // further, the code of all roles leaves the instruction cache.
        constexpr uint64_t MN = 2048 >> 4;
        const uint64_t d_k0 = sdesc(sbase + OFF_STAGE, 16, 1024), d_mn0 = sdesc(sbase + OFF_STAGE, Q * 128, 1024);
        const uint64_t d_cw0 = sdesc(sbase + OFF_CW, SZ_T, 1024), d_p0 = sdesc(sbase + OFF_P, 16, 1024);
        const uint64_t d_m0 = sdesc(sbase + OFF_M, KD * 128, 1024);
        constexpr uint64_t ST = SZ_STAGE >> 4, AB = SZ_AB >> 4, TT = SZ_T >> 4, MM = SZ_M >> 4;
        int st = 0, k3 = 0;                             // stage, turn of the ring
        if (warp == W_S && !SO) {
            for (int c = 0; c < nch; c++) {
                if (!wait(B_FULL + st, k3, 102)) break;
                if (c > 0 && !wait(B_SEMPTY, c - 1, 103)) break;
                if (chunk_n(c) < Q && !wait(B_ZERO, 0, 120)) break;     // one chunk of the walk at most
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t da = d_k0 + st * ST, db = da + AB;
                    const uint32_t d = tmem + COL_S;
#pragma unroll 1
                    for (int x = 0; x < NX; x++)
#pragma unroll
                        for (int kk = 0; kk < 4; kk++)
                            umma(d, da + x * TT + kk * 2, db + x * TT + kk * 2, id_kk, x + kk > 0);
                    umma_commit(bar(B_SFULL));
                }
                __syncwarp();
                if (++st == NST) st = 0, k3++;
            }
        } else if (warp == W_D) {
            for (int c = 0; c < nch; c++) {
                const int pb = c & 1, k2 = c >> 1;
                if (!wait(B_FULL + st, k3, 105)) break;
                if (c > 0 && !wait(B_DEMPTY, c - 1, 106)) break;
                if (!wait(B_CWFULL + pb, k2, 104)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t db = d_mn0 + st * ST + AB, dw = d_cw0 + pb * (3 * TT);
                    // the three pieces side by side in N = 192: B is read once,
                    // not three times, and the state warps add them up (forward
                    // 51 -> 50 us)
#pragma unroll
                    for (int kk = 0; kk < 4; kk++) umma(tmem + COL_D, db + kk * MN, dw + kk * MN, id_st, kk > 0);
                    umma_commit(bar(B_DFULL));
                    umma_commit(bar(B_CWEMPTY + pb));
                    umma_commit(bar(B_EMPTY + st));
                }
                __syncwarp();
                if (++st == NST) st = 0, k3++;
            }
        } else if (warp == W_Y23 && !SO) {
            for (int c = 0; c < nch; c++) {
                const int pb = c & 1, k2 = c >> 1;
                if (!wait(B_FULL + st, k3, 107)) break;
                if (c > 1 && !wait(B_YEMPTY + pb, k2 - 1, 108)) break;
                if (!wait(B_MFULL + pb, k2, 109)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t da = d_k0 + st * ST, dm = d_m0 + pb * MM;
                    const uint32_t d = tmem + COL_Y3 + pb * 64;
#pragma unroll 1
                    for (int x = 0; x < NX; x++)
#pragma unroll
                        for (int kk = 0; kk < 4; kk++)
                            umma(d, da + x * TT + kk * 2, dm + (4 * x + kk) * MN, id_kmn, x + kk > 0);
                }
                __syncwarp();
                if (!wait(B_PFULL + pb, k2, 118)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dp = d_p0 + pb * TT, dc = d_mn0 + st * ST + 2 * AB;
                    const uint32_t d = tmem + COL_Y2 + pb * 64;
#pragma unroll
                    for (int kk = 0; kk < 4; kk++) umma(d, dp + kk * 2, dc + kk * MN, id_kmn, kk > 0);
                    umma_commit(bar(B_YFULL + pb));
                    umma_commit(bar(B_EMPTY + st));
                }
                __syncwarp();
                if (++st == NST) st = 0, k3++;
            }
        }
        // every UMMA this warp issued has completed before TMEM is freed
        const int dr = B_DRAIN + warp - W_S;
        if (elect_one()) umma_commit(bar(dr));
        __syncwarp();
        const long long t0 = clock64();
        while (!mbar_try(bar(dr), 0) && clock64() - t0 < WAIT_LIMIT_CYCLES) {
        }
        __syncwarp();
    } else if (warp < W_SC) {
        // ---- Cw = w c in three bf16 pieces; rows behind the sequence zeroed in B and C
        const int wt = tid - W_CW * 32;                 // 16-byte piece wt & 7 of rows wt/8 + 16u
        const int r0 = wt >> 3;
        const f32x2 neg1 = pair(-1.f, -1.f);
        const float sw = g.scale_w;
        int st = 0, k = 0;
        for (int c = 0; c < nch; c++) {
            const int pb = c & 1, L = chunk_n(c);
            if (c > 1 && !wait(B_CWEMPTY + pb, (c >> 1) - 1, 111)) break;
            if (!wait(B_FULL + st, k, 110)) break;
            uint8_t *ct = sm + OFF_STAGE + st * SZ_STAGE + 2 * SZ_AB + wt * 16;
            if (L < Q) {
                // behind the sequence but inside the tensor B and C may hold
                // anything: zeroed before any UMMA reads this chunk
                for (int row = r0, o = 0; row < Q; row += 16, o += 2048)
                    if (row >= L) {
                        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(ct + o) = z;
#pragma unroll
                        for (int x = 1; x <= NX; x++) *reinterpret_cast<uint4 *>(ct + o - x * SZ_T) = z;
                    }
                fence_async_smem();
                arrive(B_ZERO);
            }
            uint8_t *cw = sm + OFF_CW + pb * 3 * SZ_T + wt * 16;
            const float *wp = rev ? pw + r0 + 1 : pw + (L - 1 - r0);
            const int dw = rev ? 16 : -16;
            // two rows at a time: one leaves its latencies bare, four push the
            // other roles' code out of the instruction cache
#pragma unroll 2
            for (int row = r0; row < Q; row += 16, ct += 2048, cw += 2048, wp += dw) {
                const uint4 x = *reinterpret_cast<const uint4 *>(ct);
                const float w = row < L ? *wp * sw : 0.f;
                // cut off, not rounded: the 24 bits of w c fall apart into three
                // bf16 exactly, by masks and byte moves alone
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t hs[4], ms[4], ls[4];
                const f32x2 ww = pair(w, w);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float a, b2;
                    const f32x2 v = mul2(pair(bf16_lo(xs[q]), bf16_hi(xs[q])), ww);
                    unpair(v, a, b2);
                    hs[q] = cut2(a, b2);
                    const f32x2 r = fma2(pair(cut(a), cut(b2)), neg1, v);
                    unpair(r, a, b2);
                    ms[q] = cut2(a, b2);
                    const f32x2 l = fma2(pair(cut(a), cut(b2)), neg1, r);
                    unpair(l, a, b2);
                    ls[q] = cut2(a, b2);
                }
                *reinterpret_cast<uint4 *>(cw) = make_uint4(hs[0], hs[1], hs[2], hs[3]);
                *reinterpret_cast<uint4 *>(cw + SZ_T) = make_uint4(ms[0], ms[1], ms[2], ms[3]);
                *reinterpret_cast<uint4 *>(cw + 2 * SZ_T) = make_uint4(ls[0], ls[1], ls[2], ls[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (l32 == 0) {
                mbar_arrive(bar(B_CWFULL + pb));
                mbar_arrive(bar(B_EMPTY + st));
            }
            if (++st == NST) st = 0, k++;
        }
    } else if (warp < W_ST) {
        // ---- scores: mask, round, store
        if (!SO) {
            const int q = warp & 3;                     // TMEM lane quarter: rows 16q .. 16q+15
            const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + COL_S;
            const int ra = 16 * q + (l32 >> 2), cq = 2 * (l32 & 3);
            f32x2 m[2][8];                              // the mask at this thread's places
#pragma unroll
            for (int hf = 0; hf < 2; hf++)
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int row = ra + ((e & 1) ? 8 : 0), s = 32 * hf + 8 * (e >> 1) + cq;
                    const int d0 = rev ? s - row : row - s, d1 = rev ? d0 + 1 : d0 - 1;
                    m[hf][e] = pair(d0 >= 0 ? pw[d0] * g.scale_p : 0.f, d1 >= 0 ? pw[d1] * g.scale_p : 0.f);
                }
            // stmatrix: blocks (rows 0-7, 8-15) x (column groups i, i + 1)
            const int mr = 16 * q + (l32 & 15), mc = l32 >> 4;
            const uint32_t prow = sbase + OFF_P + mr * 128;
            uint32_t po[4];
#pragma unroll
            for (int i = 0; i < 4; i++) po[i] = prow + (((2 * i + mc) ^ (mr & 7)) << 4);
            // 16 x 32 blocks wholly on the masked side are zero: written into each buffer once
            const int zhf = rev ? (q >= 2 ? 0 : 2) : (q < 2 ? 1 : 2);
            for (int c = 0; c < nch; c++) {
                const int pb = c & 1;
                if (!wait(B_SFULL, c, 112)) break;
                if (c > 1 && !wait(B_YFULL + pb, (c >> 1) - 1, 113)) break;    // P two chunks ago has been read
                tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    if (hf == zhf) {
                        if (c < 2) {
                            stmatrix4(po[2 * hf] + pb * SZ_T, 0u, 0u, 0u, 0u);
                            stmatrix4(po[2 * hf + 1] + pb * SZ_T, 0u, 0u, 0u, 0u);
                        }
                        continue;
                    }
                    float v[16];
                    uint32_t o[8];
                    tmem_ld16x256b_x4(tl + 32 * hf, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; e++) o[e] = round2(mul2(pair(v[2 * e], v[2 * e + 1]), m[hf][e]));
                    stmatrix4(po[2 * hf] + pb * SZ_T, o[0], o[1], o[2], o[3]);
                    stmatrix4(po[2 * hf + 1] + pb * SZ_T, o[4], o[5], o[6], o[7]);
                }
                tc_fence_before();
                fence_async_smem();
                __syncwarp();
                if (l32 == 0) {
                    mbar_arrive(bar(B_SEMPTY));
                    mbar_arrive(bar(B_PFULL + pb));
                }
            }
        }
    } else if (KD == 64 && warp < W_Y) {
        // ---- the state of 64 rows (an M = 64 accumulator): two rows, 32 of
        // the tile's columns in pairs, fp32
        const int q = warp & 3, c0 = 32 * ((warp - W_ST) >> 2);
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + COL_D + c0;
        const size_t elems = (size_t)g.dar * g.dcr;
        float *slots = g.ws + (size_t)lane * (g.nseg - 1) * elems;
        const int ra = 16 * q + (l32 >> 2), pc = p0 + c0 + 2 * (l32 & 3);
        f32x2 M[8];                                     // pair e: row ra + 8 (e & 1), columns 8 (e / 2) + 0, 1
        // where pair e lies in a state of global memory; a quad's four pairs
        // are 32 bytes of a row
        auto inside = [&](int e, int odd) { return ra + 8 * (e & 1) < g.dar && pc + 8 * (e >> 1) + odd < g.dcr; };
        auto at = [&](int e, int odd, bool tr) {
            const size_t n = ra + 8 * (e & 1), p = pc + 8 * (e >> 1) + odd;
            return tr ? p * g.dar + n : n * g.dcr + p;
        };
        {
            const float *src = (SO || (seg == 0 && !g.m0)) ? nullptr
                               : (seg == 0 ? g.m0 + lane * elems : slots + (size_t)(seg - 1) * elems);
            const bool tr = seg == 0 && g.m_trans;
#pragma unroll
            for (int e = 0; e < 8; e++) M[e] = 0ull;
            if (src) {
                // all sixteen loads go out before one is looked at: those outside
                // the state read its last element
                const size_t last = elems - 1;
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; e++) x[e] = src[inside(e >> 1, e & 1) ? at(e >> 1, e & 1, tr) : last];
#pragma unroll
                for (int e = 0; e < 8; e++)
                    M[e] = pair(inside(e, 0) ? x[2 * e] : 0.f, inside(e, 1) ? x[2 * e + 1] : 0.f);
            }
        }
        const int mr = 16 * q + (l32 & 15), mc = l32 >> 4;
        uint32_t mo[2];
#pragma unroll
        for (int i = 0; i < 2; i++) mo[i] = sbase + OFF_M + mr * 128 + (((c0 / 8 + 2 * i + mc) ^ (mr & 7)) << 4);
        auto publish = [&](int buf) {                   // the rounded copy that D3 reads
            stmatrix4(mo[0] + buf * SZ_M, round2(M[0]), round2(M[1]), round2(M[2]), round2(M[3]));
            stmatrix4(mo[1] + buf * SZ_M, round2(M[4]), round2(M[5]), round2(M[6]), round2(M[7]));
            fence_async_smem();
            arrive(B_MFULL + buf);
        };
        if (!SO && nch > 0) publish(0);
        for (int c = 0; c < nch; c++) {
            const int pb = c & 1;
            const Decay d = decay_of(pw[chunk_n(c)], pm1[chunk_n(c)]);
            const f32x2 keep = pair(d.keep, d.keep), df = pair(d.f, d.f);
            if (!wait(B_DFULL, c, 114)) break;
            tc_fence_after();
            float hi[16], mid[16], lo[16];
            tmem_ld16x256b_x4(tl, hi);
            tmem_ld16x256b_x4(tl + 64, mid);
            tmem_ld16x256b_x4(tl + 128, lo);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const f32x2 s = add2(add2(pair(lo[2 * e], lo[2 * e + 1]), pair(mid[2 * e], mid[2 * e + 1])),
                                     pair(hi[2 * e], hi[2 * e + 1]));
                M[e] = fma2(M[e], keep, fma2(M[e], df, s));
            }
            tc_fence_before();
            arrive(B_DEMPTY);
            if (!SO && c + 1 < nch) {
                // buffer (c+1) & 1 was last read by D3 of chunk c - 1
                if (c > 0 && !wait(B_YFULL + (pb ^ 1), (c - 1) >> 1, 115)) break;
                publish(pb ^ 1);
            }
        }
        float *dst = SO ? slots + (size_t)seg * elems
                        : (seg == g.nseg - 1 && g.m_out ? g.m_out + lane * elems : nullptr);
        if (dst && !*abort_flag) {
            const bool tr = !SO && g.m_trans;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                float a, b2;
                unpair(M[e], a, b2);
                if (inside(e, 0)) dst[at(e, 0, tr)] = a;
                if (inside(e, 1)) dst[at(e, 1, tr)] = b2;
            }
        }
    } else if (KD == 128 && warp < W_Y) {
        // ---- the state: this thread's row, 32 of the tile's columns, fp32
        const int q = warp & 3, n = 32 * q + l32, ch = (warp - W_ST) >> 2, c0 = 32 * ch;
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + COL_D + c0;
        const size_t elems = (size_t)g.dar * g.dcr;
        float *slots = g.ws + (size_t)lane * (g.nseg - 1) * elems;
        const bool mine = n < g.dar;
        f32x2 M[16];
        // fp32 states go to and from global memory by way of this warp's 32 rows
        // of the M buffers, as fp32 rows of 128 bytes (16-byte pieces XOR row):
        // a thread's own row is a scattered access, four rows a warp are not
        uint8_t *stg = sm + OFF_M + (q * 2 + ch) * 4096;
        auto piece = [&](int row, int k) { return reinterpret_cast<float4 *>(stg + row * 128 + ((k ^ (row & 7)) << 4)); };
        const int wr = l32 >> 3, wk = l32 & 7;          // row of four, 16-byte piece
        const bool in = p0 + c0 + 4 * wk < g.dcr;
        // element by element where the state is transposed or its rows are no
        // whole 16-byte pieces
        auto at = [&](int p, bool tr) { return tr ? (size_t)(p0 + c0 + p) * g.dar + n : (size_t)n * g.dcr + p0 + c0 + p; };
        const bool pieces = g.dcr % 4 == 0;
        {
            const float *src = (SO || (seg == 0 && !g.m0)) ? nullptr
                               : (seg == 0 ? g.m0 + lane * elems : slots + (size_t)(seg - 1) * elems);
#pragma unroll
            for (int p = 0; p < 16; p++) M[p] = 0ull;
            const bool tr = seg == 0 && g.m_trans;
            if (src && (tr || !pieces)) {
                const size_t last = elems - 1;          // as in the 64-wide variant
                float x[32];
#pragma unroll
                for (int p = 0; p < 32; p++) x[p] = src[mine && p0 + c0 + p < g.dcr ? at(p, tr) : last];
#pragma unroll
                for (int p = 0; p < 32; p += 2)
                    M[p / 2] = pair(mine && p0 + c0 + p < g.dcr ? x[p] : 0.f, mine && p0 + c0 + p + 1 < g.dcr ? x[p + 1] : 0.f);
            } else if (src) {
#pragma unroll 4
                for (int r = wr; r < 32; r += 4) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in && 32 * q + r < g.dar)
                        v = *reinterpret_cast<const float4 *>(src + (size_t)(32 * q + r) * g.dcr + p0 + c0 + 4 * wk);
                    *piece(r, wk) = v;
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float4 v = *piece(l32, k);
                    M[2 * k] = pair(v.x, v.y);
                    M[2 * k + 1] = pair(v.z, v.w);
                }
                // the other warps' rows are in the buffers that publish() writes:
                // meet here (every state warp takes this branch together)
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
        }
        auto publish = [&](int buf) {                   // the rounded copy that D3 reads
            uint8_t *mt = sm + OFF_M + buf * SZ_M + n * 128;
#pragma unroll
            for (int k = 0; k < 4; k++)
                *reinterpret_cast<uint4 *>(mt + (((4 * ch + k) ^ (n & 7)) << 4)) =
                    make_uint4(round2(M[4 * k]), round2(M[4 * k + 1]), round2(M[4 * k + 2]), round2(M[4 * k + 3]));
            fence_async_smem();
            arrive(B_MFULL + buf);
        };
        if (!SO && nch > 0) publish(0);
        for (int c = 0; c < nch; c++) {
            const int pb = c & 1;
            const Decay d = decay_of(pw[chunk_n(c)], pm1[chunk_n(c)]);
            const f32x2 keep = pair(d.keep, d.keep), df = pair(d.f, d.f);
            if (!wait(B_DFULL, c, 114)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; k++) {
                float hi[8], mid[8], lo[8];
                tmem_ld8(tl + 8 * k, hi);
                tmem_ld8(tl + 64 + 8 * k, mid);
                tmem_ld8(tl + 128 + 8 * k, lo);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const f32x2 s = add2(add2(pair(lo[2 * u], lo[2 * u + 1]), pair(mid[2 * u], mid[2 * u + 1])),
                                         pair(hi[2 * u], hi[2 * u + 1]));
                    M[4 * k + u] = fma2(M[4 * k + u], keep, fma2(M[4 * k + u], df, s));
                }
            }
            tc_fence_before();
            arrive(B_DEMPTY);
            if (!SO && c + 1 < nch) {
                // buffer (c+1) & 1 was last read by D3 of chunk c - 1
                if (c > 0 && !wait(B_YFULL + (pb ^ 1), (c - 1) >> 1, 115)) break;
                publish(pb ^ 1);
            }
        }
        float *dst = SO ? slots + (size_t)seg * elems
                        : (seg == g.nseg - 1 && g.m_out ? g.m_out + lane * elems : nullptr);
        bool out = dst && !*abort_flag;
        // the last chunk's D3 still reads the buffers
        const bool tro = !SO && g.m_trans, single = tro || !pieces;
        if (out && !SO && !single && nch > 0) out = wait(B_YFULL + ((nch - 1) & 1), (nch - 1) >> 1, 121);
        if (out && single) {
            if (mine) {
#pragma unroll
                for (int p = 0; p < 32; p += 2) {
                    float a, b2;
                    unpair(M[p / 2], a, b2);
                    if (p0 + c0 + p < g.dcr) dst[at(p, tro)] = a;
                    if (p0 + c0 + p + 1 < g.dcr) dst[at(p + 1, tro)] = b2;
                }
            }
        } else if (out) {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                float4 v;
                unpair(M[2 * k], v.x, v.y);
                unpair(M[2 * k + 1], v.z, v.w);
                *piece(l32, k) = v;
            }
            __syncwarp();
#pragma unroll 4
            for (int r = wr; r < 32; r += 4)
                if (in && 32 * q + r < g.dar)
                    *reinterpret_cast<float4 *>(dst + (size_t)(32 * q + r) * g.dcr + p0 + c0 + 4 * wk) = *piece(r, wk);
        }
    } else if (!SO && g.y) {
        // ---- the answers
        const int q = warp & 3, wy = warp - W_Y;
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        const int ra = 16 * q + (l32 >> 2), rb = ra + 8, cq = 2 * (l32 & 3);
        const int mr = l32 & 15, mc = l32 >> 4;         // stmatrix rows, as for the scores
        const uint32_t ybase = sbase + OFF_Y + 16 * q * 128;   // this warp's 16 rows
        uint32_t yo[4];
#pragma unroll
        for (int i = 0; i < 4; i++) yo[i] = ybase + mr * 128 + (((2 * i + mc) ^ (mr & 7)) << 4);
        const float si = g.scale_i;
        // y goes by way of shared memory: from there by TMA, 64 columns of bf16
        // or 32 of fp32 (whose stores from registers, 32 bytes of a row each, took
        // 254 us where these take 170: 8 x 2048 tokens, 16 heads over 4 groups, dq
        // and dk), or by its elements where bf16 rows are no whole 16-byte pieces
        const bool f32 = g.y_f32, tma = f32 || g.dcr == g.dc;
        __nv_bfloat16 *yh = static_cast<__nv_bfloat16 *>(g.y) + ((b * g.T + t_beg) * g.H + h) * g.dcr + p0;
        auto store = [&](int col, int64_t t) {          // the staged rows, as rows t of y
            if (l32 == 0 && p0 + col < g.dc && t < g.T) tma_store4(&P.my[pi], p0 + col, (int)h, (int)t, (int)b, ybase);
        };
        for (int c = 0; c < nch; c++) {
            const int pb = c & 1, L = chunk_n(c), t = chunk_t(c);
            if (!wait(B_YFULL + pb, c >> 1, 116)) break;
            tc_fence_after();
            const float fa = ra < L ? pw[rev ? L - 1 - ra : ra + 1] * si : 0.f;
            const float fb = rb < L ? pw[rev ? L - 1 - rb : rb + 1] * si : 0.f;
            const f32x2 fa2 = pair(fa, fa), fb2 = pair(fb, fb);
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                float y2[16], y3[16];
                f32x2 o[8];
                tmem_ld16x256b_x4(tl + COL_Y2 + pb * 64 + 32 * hf, y2);
                tmem_ld16x256b_x4(tl + COL_Y3 + pb * 64 + 32 * hf, y3);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; e++)
                    o[e] = fma2((e & 1) ? fb2 : fa2, pair(y3[2 * e], y3[2 * e + 1]), pair(y2[2 * e], y2[2 * e + 1]));
                if (L < Q) {                            // rows behind the sequence are zeros
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (((e & 1) ? rb : ra) >= L) o[e] = 0ull;
                }
                if (f32 || hf == 0) {                   // what was staged before is on its way
                    if (l32 == 0) tma_store_wait_read();
                    __syncwarp();
                }
                if (!f32) {
                    stmatrix4(yo[2 * hf], round2(o[0]), round2(o[1]), round2(o[2]), round2(o[3]));
                    stmatrix4(yo[2 * hf + 1], round2(o[4]), round2(o[5]), round2(o[6]), round2(o[7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int r = (l32 >> 2) + 8 * (e & 1), k = 2 * (e >> 1) + ((l32 >> 1) & 1);
                        *reinterpret_cast<f32x2 *>(sm + OFF_Y + (16 * q + r) * 128 + ((k ^ (r & 7)) << 4) + 8 * (l32 & 1)) = o[e];
                    }
                    fence_async_smem();
                    __syncwarp();
                    store(32 * hf, t_beg + t + 16 * q);
                }
            }
            tc_fence_before();
            fence_async_smem();
            __syncwarp();
            if (l32 == 0) mbar_arrive(bar(B_YEMPTY + pb));
            if (!f32 && tma) store(0, t_beg + t + 16 * q);
            __syncwarp();
            if (!tma) {
                // row by row, in pairs where a row is whole pairs
                const int64_t left = g.T - (t_beg + t + 16 * q), step = (int64_t)g.H * g.dcr;
                const int rows = left < 16 ? (int)left : 16, cols = g.dcr - p0;
                __nv_bfloat16 *out = yh + (t + 16 * q) * step;
                const uint8_t *in = sm + OFF_Y + 16 * q * 128;
                auto piece = [&](int r, int p) { return in + r * 128 + (((p >> 3) ^ (r & 7)) << 4) + 2 * (p & 7); };
                if (g.dcr % 2 == 0) {
#pragma unroll 4
                    for (int r = 0; r < rows; r++)
                        if (2 * l32 < cols)
                            *reinterpret_cast<uint32_t *>(out + r * step + 2 * l32) =
                                *reinterpret_cast<const uint32_t *>(piece(r, 2 * l32));
                } else {
#pragma unroll 2
                    for (int r = 0; r < rows; r++) {
                        if (l32 < cols) out[r * step + l32] = *reinterpret_cast<const __nv_bfloat16 *>(piece(r, l32));
                        if (l32 + 32 < cols)
                            out[r * step + l32 + 32] = *reinterpret_cast<const __nv_bfloat16 *>(piece(r, l32 + 32));
                    }
                }
                __syncwarp();
            }
        }
        // rows behind the sequence in the segment's chunks that were not walked:
        // zeros, 16 rows a store (8 x 2048 tokens, 16 heads, 100 tokens each:
        // 70 us with one row a warp and store)
        const int64_t z0 = t_beg + (int64_t)nch * Q, e = t_beg + g.seg_len < g.T ? t_beg + g.seg_len : g.T;
        if (z0 < e && tma) {
            if (l32 == 0) tma_store_wait_read();
            __syncwarp();
            for (int v = l32; v < 128; v += 32)
                *reinterpret_cast<uint4 *>(sm + OFF_Y + 16 * q * 128 + 16 * v) = make_uint4(0u, 0u, 0u, 0u);
            fence_async_smem();
            __syncwarp();
            for (int64_t t = z0 + 16 * q; t < e; t += 64) {
                store(0, t);
                if (f32) store(32, t);
            }
        } else {
            uint16_t *row = static_cast<uint16_t *>(g.y) + ((b * g.T + z0 + wy) * g.H + h) * g.dcr + p0 + l32;
            const int left = g.dcr - p0 - l32;
            const int64_t step = 4 * g.H * g.dcr;
#pragma unroll 4
            for (int64_t t = z0 + wy; t < e; t += 4, row += step) {
                if (left > 0) row[0] = 0;
                if (left > 32) row[32] = 0;
            }
        }
        if (l32 == 0) tma_store_wait_all();
    } else if (!SO) {
        // no answer is wanted, only the state: hand the accumulators back
        for (int c = 0; c < nch; c++) {
            if (!wait(B_YFULL + (c & 1), c >> 1, 117)) break;
            arrive(B_YEMPTY + (c & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_S) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

__device__ int g_error;

// ---- host side -------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// bf16 (or fp32) rows (Bt, T, heads, d) with ld elements from token to token:
// boxes of 128 bytes of `rows` tokens, zeros outside
static bool rows_map(CUtensorMap *m, const void *base, int64_t d, int64_t heads, int64_t T, int64_t Bt, int64_t ld,
                     uint32_t rows, bool f32 = false) {
    const int64_t size = f32 ? 4 : 2;
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)Bt};
    const cuuint64_t strides[3] = {(cuuint64_t)(d * size), (cuuint64_t)(ld * size), (cuuint64_t)(ld * T * size)};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / size), 1, rows, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mixtc

// Up to 256 lanes of up to 16 tokens are one block each of the fp32 kernel, for
// its exactness: a few tokens behind a prompt are then as exact as single steps.  It
// costs little: 128 x 64 states, 16 tokens there against 17 here, forward and
// backward, replayed with a cold L2: 16 lanes 12.3 and 18.5 us against 10.3 and
// 20.5, 256 lanes 22.5 and 59.4 against 18.4 and 60.  With 1024 lanes it would be
// a fifth more (forward 61 us there, 49 here).
bool mix_tc_sizes(const MixArgs &g, m3_dtype dt) {
    if (dt != M3_BF16 || g.da > mixtc::DA || g.dc > mixtc::DA || g.da % 8 || g.dc % 8 || g.T < 1) return false;
    if (g.T <= 16 && g.Bt * g.H <= 256) return false;
    if (g.Bt * g.H > (int64_t)1 << 28) return false;      // three problems of two column tiles share a 1-D grid
    // a TMA stride is a multiple of 16 bytes below 2^40
    for (int64_t ld : {g.lda, g.ldb, g.ldc, 2 * g.H * g.dc})
        if (ld % 8 || ld > ((int64_t)1 << 38) / g.T) return false;
    return true;
}

static int padded(const MixArgs &g) { return g.da <= 64 ? 64 : 128; }

// Segments of the problems of one launch (those padded to the same width; the
// same count for all).  A CTA holds an SM, so k CTAs take ceil(k / 148) waves.
// A wave takes its chunks and about 4 chunks' time more (set-up, the first
// loads, the last chunk's way through the roles: 5 us); the state pass over
// the leading segments takes half a chunk's time per chunk.  The count with the
// least time in those units, at least 4 chunks a segment, at most 64 segments
// and 64 MB of states.  (1 x 32768 tokens, 32 heads: 357 us with 32 segments,
// which a rule without the fixed part takes.)
static void plan_width(MixArgs *g, int n, int kd) {
    using namespace mixtc;
    const int64_t nq = (g[0].T + Q - 1) / Q;
    int64_t ctas = 0, state = 0;
    for (int i = 0; i < n; i++) {
        if (padded(g[i]) != kd) continue;
        ctas += g[i].Bt * g[i].H * ((g[i].dc + DC - 1) / DC);
        state += g[i].Bt * g[i].H * g[i].dar * g[i].dcr * 4;
        g[i].nseg = 1;
        g[i].seg_len = (nq > 0 ? nq : 1) * Q;
    }
    if (ctas == 0 || ctas >= 148 || nq < 8) return;
    const int64_t most = ((int64_t)64 << 20) / state;
    auto waves = [](int64_t k) { return (k + 147) / 148; };
    double best = (double)waves(ctas) * (double)(nq + 4);
    for (int64_t ns = 2; ns <= 64; ns++) {
        const int64_t len = (nq + ns - 1) / ns;
        if (len < 4) break;
        const int64_t k = (nq + len - 1) / len;
        if (k < 2 || k - 1 > most) continue;
        const double cost = (double)waves(ctas * k) * (double)(len + 4) + (double)waves(ctas * (k - 1)) * (0.5 * (double)len + 4);
        if (cost < best - 1e-9) {
            best = cost;
            for (int i = 0; i < n; i++)
                if (padded(g[i]) == kd) {
                    g[i].nseg = (int)k;
                    g[i].seg_len = len * Q;
                }
        }
    }
}
void mix_tc_plan(MixArgs *g, int n) {
    plan_width(g, n, 64);
    plan_width(g, n, 128);
}

// What a launch needs of its device, looked up once per device: the kernels'
// shared-memory size set, the error word's address.
template <int KD>
static cudaError_t set_smem() {
    using namespace mixtc;
    const cudaError_t e = cudaFuncSetAttribute(k_mix_tc<true, KD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<KD>::SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(k_mix_tc<false, KD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<KD>::SMEM);
}
static cudaError_t device_setup(int **err) {
    static std::atomic<int *> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*err = known[dev].load(std::memory_order_acquire))) return cudaSuccess;
    if ((e = set_smem<64>()) != cudaSuccess || (e = set_smem<128>()) != cudaSuccess ||
        (e = cudaGetSymbolAddress(reinterpret_cast<void **>(err), mixtc::g_error)) != cudaSuccess)
        return e;
    if (dev < 64) known[dev].store(*err, std::memory_order_release);
    return cudaSuccess;
}

template <bool SO>
static cudaError_t launch_pass(mixtc::Batch &P, int kd, cudaStream_t s) {
    using namespace mixtc;
    unsigned k = 0;
    for (int i = 0; i < P.n; i++) {
        P.first[i] = k;
        k += (unsigned)(P.g[i].Bt * P.g[i].H * (P.g[i].nseg - (SO ? 1 : 0)) * ((P.g[i].dc + DC - 1) / DC));
    }
    P.first[P.n] = k;
    if (kd == 64) k_mix_tc<SO, 64><<<k, THREADS, Lay<64>::SMEM, s>>>(P);
    else k_mix_tc<SO, 128><<<k, THREADS, Lay<128>::SMEM, s>>>(P);
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_mix_tc(const MixArgs *g, int n, cudaStream_t s) {
    using namespace mixtc;
    Batch P;
    cudaError_t e = device_setup(&P.err);
    if (e != cudaSuccess) return e;
    for (int kd : {64, 128}) {
        P.n = 0;
        bool split = false;
        for (int i = 0; i < n; i++) {
            const MixArgs &a = g[i];
            if (padded(a) != kd) continue;
            if (P.n == MAXP) return cudaErrorInvalidValue;
            const int k = P.n++;
            if (!rows_map(&P.ma[k], a.a, a.da, a.H / a.ra, a.T, a.Bt, a.lda, Q) ||
                !rows_map(&P.mb[k], a.b, a.da, a.H / a.rb, a.T, a.Bt, a.ldb, Q) ||
                !rows_map(&P.mc[k], a.c, a.dc, a.H / a.rc, a.T, a.Bt, a.ldc, Q) ||
                (a.y && (a.y_f32 || a.dcr == a.dc) &&
                 !rows_map(&P.my[k], a.y, a.dc, a.H, a.T, a.Bt, a.H * a.dc, 16, a.y_f32)))
                return cudaErrorInvalidValue;
            P.g[k] = a;
            split |= a.nseg > 1;
        }
        if (P.n == 0) continue;
        if (split) {
            if ((e = launch_pass<true>(P, kd, s)) != cudaSuccess) return e;
            if ((e = launch_mix_combine(P.g, P.n, s)) != cudaSuccess) return e;
        }
        if ((e = launch_pass<false>(P, kd, s)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

int mix_tc_error_and_clear(cudaStream_t s) {
    int *err = nullptr, v = 0;
    const int zero = 0;
    if (cudaGetSymbolAddress(reinterpret_cast<void **>(&err), mixtc::g_error) != cudaSuccess) return -1;
    if (cudaMemcpyAsync(&v, err, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return -1;
    if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    if (v) {
        if (cudaMemcpyAsync(err, &zero, sizeof(int), cudaMemcpyHostToDevice, s) != cudaSuccess) return -1;
        if (cudaStreamSynchronize(s) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace m3

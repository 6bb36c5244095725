// minikv_window_prefill: prompt attention with a sliding window and sinks.
//
// Query row i of Tq stands at position p = Tk - Tq + i and sees the keys
// j <= p with p - j < window, and the keys j < n_sink.  Only the 128-key blocks
// that hold a visible key are read: the sink blocks, then the band.
//
// One CTA = two 128-row query tiles of one (sequence, KV head): the KV head's
// tiles are numbered (position tile, query head of the group), heads fastest,
// and CTA c takes tiles 2c and 2c + 1, so an even group shares every K / V
// block between two heads at the same positions.  12 warps:
//   warp 0      TMA producer: both Q tiles, then K_0, V_0, K_1, V_1, .. into a
//               ring of 5 x 32 KB;
//   warp 1      TMEM owner;
//   warps 2, 3  issue tcgen05.mma, a warp a query tile;
//   warps 4-7   softmax of tile 0, warps 8-11 of tile 1: thread = query row =
//               TMEM lane; also the rescale of O and the epilogue.
// Tensor memory (all 512 columns): S_0, S_1, O_0, O_1 fp32 [128 x 128].  P_t
// (fp16 pairs, 64 columns) takes the place of S_t once the row is in registers.
// Issue order of tile t: S(0), then for every block j P V(j), S(j+1): while a
// tile's softmax works, the tensor cores have the other tile's two products.
// One warp issuing for both tiles left the pipe idle during its waits (about 250
// cycles each under running MMAs, 1100 of 4400 a block pair).  A commit covers
// everything its thread issued before it, so S_t(j+1) complete means O_t holds
// block j: the softmax may rescale O_t.  tcgen05.mma of one thread run in issue
// order, so S_t(j+1) over P_t(j) is safe.
//
// Softmax: base 2, running reference max that moves only when a score passes it
// by 2^8 (p <= 256 keeps its 11 bits in fp16; O is rescaled rarely).  P is
// rounded to fp16 for the tensor cores (2^-12 relative a term on average, the
// precision of the output); the sum is taken in fp32 before that rounding.
// Hidden keys are -inf before the max, and the reference starts at a finite
// -1e30, so a block without a visible key for a row leaves that row as it was.
//
// A hidden key's value row meets P = 0 in the tensor cores, and 0 times an
// infinity or NaN is NaN, which stays in O.  So a warp with rows whose weights are
// finite and whose output is not looks at the values once (explain_rows): channels
// that meet such a value among the row's visible keys get what the sum gives, and
// only rows with others left are computed again, by slow_row (CUDA cores, visible
// keys only).  8192 tokens, 32 heads, window 4096: 0.43 ms; with a NaN in a sink,
// which all rows see, 0.95 (computed again row by row 66); with NaN padding behind
// 8100 tokens 12, for the 36 rows a head that share a block with it.
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "tc.cuh"

namespace minikv {

namespace {

constexpr int kM = 128, kN = 128;          // query rows of a tile, keys of a block
constexpr int kRing = 5;                    // K / V blocks in flight
constexpr int kThreads = 384;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 t
// Keys taken of a block of sinks that has no more (a handful is usual): 512 tokens, window 128 take 8.5 us instead of
// 9.4 with the whole block, 2 x 3001 tokens, window 1000 147 instead of 149.
constexpr int kFew = 32;
constexpr float kLazy = 8.f;
constexpr float kNone = -1e30f;             // reference max of a row that has seen nothing

struct Smem {
    uint16_t q[2][2][kM * 64];       // [tile][64-wide d block], 128-byte swizzle
    uint16_t kv[kRing][2][kN * 64];
    // mbarriers, initialised by kBars lanes at once
    uint64_t q_full, full[kRing];
    uint64_t done[2];                // step 0, S(0), and j + 1, P V(j) and S(j + 1), of every tile have read their blocks
    uint64_t p_full[2], s_full[2], o_done[2], drain[2];
    uint32_t tmem_base;
    int abort;
};

struct Args {
    const uint16_t *q, *k, *v;
    unsigned *status;   // one word a query tile: 1 = a bounded wait expired, its outputs are not valid
    int Hq, Hkv, Tq, Tk, window, n_sink;
    int units, ncta, ntile, per;   // B * Hkv; CTAs and query tiles of a unit, tiles of a CTA (1 or 2)
    float scale_log2;
};

__device__ __forceinline__ bool wait_warp(Smem &s, uint64_t *bar, uint32_t parity) {
    return tc::role_wait_warp(&s.abort, bar, parity);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// bits [lo, hi) of a 32-bit word, any int lo, hi
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
    const uint32_t below_hi = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1;
    const uint32_t below_lo = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1;
    return below_hi & ~below_lo;
}

// One query tile: query head, first query row, and the rows' first and last position.
struct Tile {
    int h, q0, p0, p1;
};
__device__ __forceinline__ Tile tile_of(const Args &a, int kvh, int i) {
    const int g = a.Hq / a.Hkv, pt = i / g;
    Tile t;
    t.h = kvh * g + i - pt * g;
    t.q0 = pt * kM;
    t.p0 = a.Tk - a.Tq + t.q0;
    t.p1 = min(t.p0 + kM - 1, a.Tk - 1);
    return t;
}
// The CTA's key blocks: n_s sink blocks, then band blocks lo .. hi.
struct Blocks {
    int n_s, lo, n;
    __device__ __forceinline__ int at(int j) const { return j < n_s ? j : lo + j - n_s; }
};
__device__ __forceinline__ Blocks blocks_of(const Args &a, int p0, int p1) {
    Blocks b;
    b.lo = max(0, p0 - (a.window - 1)) / kN;
    b.n_s = min(b.lo, (int)(((long long)a.n_sink + kN - 1) / kN));
    b.n = b.n_s + p1 / kN - b.lo + 1;
    return b;
}

// One query row from scratch over its visible keys (fp32, a warp a row, a lane
// four channels), eight keys at a time: the row at position p into its place in
// the swizzled output tile, dst its first byte there.
__device__ __forceinline__ void slow_row(const Args &a, size_t qrow, size_t kvplane, int p, unsigned char *dst, int sw,
                                         int lane) {
    constexpr int kKeys = 8;
    const int lo = max(0, p - (a.window - 1)), ns = min(a.n_sink, lo), n = ns + p - lo + 1;
    auto quad = [&](const uint16_t *row, float (&f)[4]) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(row) + lane);
        const float2 x = unpack_half2(u.x), y = unpack_half2(u.y);
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    };
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    quad(a.q + qrow * kD, q);
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += kKeys) {
        float x[kKeys], v[kKeys][4], top = m;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const int t = min(t0 + i, n - 1);
            const size_t j = kvplane * a.Tk + (t < ns ? t : lo + t - ns);
            float k[4];
            quad(a.k + j * kD, k);
            quad(a.v + j * kD, v[i]);
            x[i] = fmaf(q[3], k[3], fmaf(q[2], k[2], fmaf(q[1], k[1], q[0] * k[0])));
        }
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
#pragma unroll
            for (int s = 16; s; s >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], s);
            x[i] = t0 + i < n ? x[i] * a.scale_log2 : -INFINITY;
            top = fmaxf(top, x[i]);
        }
        const float al = m == top ? 1.f : ex2(m - top);
        m = top;
        l *= al;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] *= al;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            if (x[i] == -INFINITY) continue;   // (the same for the whole warp)
            const float e = ex2(x[i] - m);
            l += e;
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = fmaf(e, v[i][c], o[c]);
        }
    }
    const float inv = 1.f / l;
    const int ch = lane >> 1;   // as the epilogue writes it: 16-byte chunk ch of the row, in halves
    *reinterpret_cast<uint2 *>(dst + (ch >> 3) * (kM * 128) + (((ch & 7) ^ sw) << 4) + 8 * (lane & 1)) =
        make_uint2(pack_half2(o[0] * inv, o[1] * inv), pack_half2(o[2] * inv, o[3] * inv));
}

// The warp's rows (mask `bad`, of row p0 + bit) whose output is not finite, put right: one look at the values of the
// CTA's blocks tells, for all 32 rows at once, which of a row's channels meet a NaN or an infinity among the keys the
// row sees.  Those channels are what the sum gives (every weight is positive): NaN, or the infinity.  Only rows with
// another channel that is not finite, spoilt by a key they do not see, are computed again; their mask is returned.
// A lane has eight channels of every second key.  tile: the warp's rows of the output tile.
__device__ __forceinline__ uint32_t explain_rows(const Args &a, const Blocks &blk, bool few, size_t kvplane, int p0,
                                                 uint32_t bad, unsigned char *tile, int lane) {
    constexpr int kLoads = 16;
    const int ch = lane & 15, odd = lane >> 4, p = p0 + lane;
    uint32_t nan[8], pos[8], neg[8];   // rows that see such a value in the lane's channel i
#pragma unroll
    for (int i = 0; i < 8; ++i) nan[i] = pos[i] = neg[i] = 0;
    auto half = [](const uint4 &v, int i) {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return (i & 1 ? w >> 16 : w) & 0xFFFFu;
    };
    auto odd_one = [](uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; };   // a half not finite?
    auto odd_ones = [&](const uint4 &v) { return odd_one(v.x) | odd_one(v.y) | odd_one(v.z) | odd_one(v.w); };
#pragma unroll 1
    for (int j = 0; j < blk.n; ++j) {
        const int k0 = blk.at(j) * kN, k1 = min(k0 + (few && j == 0 ? kFew : kN), a.Tk);
#pragma unroll 1
        for (int k = k0; k < k1; k += 2 * kLoads) {
            uint4 v[kLoads];
            uint32_t any = 0;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = min(k + 2 * u + odd, k1 - 1);
                v[u] = __ldg(reinterpret_cast<const uint4 *>(a.v + (kvplane * a.Tk + key) * kD) + ch);
                any |= odd_ones(v[u]);
            }
            if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                if (!__any_sync(0xffffffffu, odd_ones(v[u]))) continue;
                uint32_t see[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = min(k + 2 * u + e, k1 - 1);
                    see[e] = __ballot_sync(0xffffffffu, key <= p && (p - key < a.window || key < a.n_sink));
                }
                const uint32_t rows = odd ? see[1] : see[0];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t x = half(v[u], i);
                    if ((x & 0x7FFFu) > 0x7C00u) nan[i] |= rows;
                    if (x == 0x7C00u) pos[i] |= rows;
                    if (x == 0xFC00u) neg[i] |= rows;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        nan[i] |= __shfl_xor_sync(0xffffffffu, nan[i], 16);
        pos[i] |= __shfl_xor_sync(0xffffffffu, pos[i], 16);
        neg[i] |= __shfl_xor_sync(0xffffffffu, neg[i], 16);
    }
    uint32_t again = 0;
    for (; bad; bad &= bad - 1) {
        const int r = __ffs(bad) - 1;
        uint4 *at = reinterpret_cast<uint4 *>(tile + (ch >> 3) * (kM * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
        const uint4 o = *at;
        uint32_t h[8], left = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = half(o, i);
            if ((nan[i] | (pos[i] & neg[i])) >> r & 1) h[i] = 0x7FFFu;
            else if (pos[i] >> r & 1) h[i] = 0x7C00u;
            else if (neg[i] >> r & 1) h[i] = 0xFC00u;
            else if ((h[i] & 0x7C00u) == 0x7C00u) left = 1;
        }
        if (__any_sync(0xffffffffu, left)) again |= 1u << r;
        __syncwarp();
        if (!odd) *at = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    __syncwarp();
    return again;
}

__global__ void __launch_bounds__(kThreads, 1)
    window_fa_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                     const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem &s = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
    // (broadcast: the compiler then knows that branches on the warp, and descriptors behind them, are uniform)
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

    // the tiles with the longest bands first, all units side by side: their K / V bands overlap in L2
    const int first = (a.ncta - 1 - (int)blockIdx.x / a.units) * a.per, unit = (int)blockIdx.x % a.units;
    const int b = unit / a.Hkv, kvh = unit - b * a.Hkv;
    const Tile t0 = tile_of(a, kvh, first);
    const bool two = a.per == 2 && first + 1 < a.ntile;   // else tile 1's warps have nothing to do
    const Tile t1 = two ? tile_of(a, kvh, first + 1) : t0;
    const Blocks blk = blocks_of(a, min(t0.p0, t1.p0), max(t0.p1, t1.p1));

    // the first block is one of sinks, few of them, which every row sees: only kFew of its keys are multiplied
    const bool few = blk.n_s == 1 && a.n_sink <= kFew;

    constexpr int kBars = 1 + kRing + 10;
    if (warp == 0) {
        const int i = lane - (1 + kRing);
        if (lane < kBars) mbar_init(&s.q_full + lane, i < 0 || i > 3 ? 1 : i > 1 ? 4 : two ? 2 : 1);   // done: issuers; p_full: warps
        fence_mbar_init();
        if (lane == 0) s.abort = 0;
    }
    if (warp == 1) tc::tmem_alloc(&s.tmem_base, 512);
    // A programmatic dependent of the work before it: the set-up above may run under that work's tail, every
    // access to global memory comes after this wait.
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem_base, 0);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
        if (warp == 0 && lane == 0) {
            // ---------------- producer
            tc::prefetch_map(&map_q);
            tc::prefetch_map(&map_k);
            tc::prefetch_map(&map_v);
            mbar_arrive_expect_tx(&s.q_full, (two ? 4 : 2) * kM * 128);
            for (int t = 0; t < (two ? 2 : 1); ++t) {
                const Tile &ti = t ? t1 : t0;
                tc::tma_load_3d(s.q[t][0], &map_q, 0, ti.q0, b * a.Hq + ti.h, &s.q_full);
                tc::tma_load_3d(s.q[t][1], &map_q, 64, ti.q0, b * a.Hq + ti.h, &s.q_full);
            }
            // K_j and V_j take the slots of V_{j-3} and K_{j-2}, both free after step j - 2 (of the two barriers that
            // count steps, the one waited on moves again with step j, which needs K_j)
            int issued = 0;
            for (int j = 0; j < blk.n; ++j) {
                if (j >= 2 && !tc::role_wait(&s.abort, &s.done[j & 1], ((j - 2) >> 1) & 1)) break;
                const int row = blk.at(j) * kN;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int st = (2 * j + v) % kRing;
                    const CUtensorMap *m = v ? &map_v : &map_k;
                    mbar_arrive_expect_tx(&s.full[st], 2 * kN * 128);
                    tc::tma_load_3d(s.kv[st][0], m, 0, row, unit, &s.full[st]);
                    tc::tma_load_3d(s.kv[st][1], m, 64, row, unit, &s.full[st]);
                }
                issued = 2 * j + 2;
            }
            // Every load queued here lands before the CTA exits, whoever gave up and whenever: another role may abort
            // after any look at s.abort.  (Without an abort these phases are long over, or about to be.)
            mbar_wait(&s.q_full, 0);
            for (int e = issued > kRing ? issued - kRing : 0; e < issued; ++e)
                mbar_wait(&s.full[e % kRing], (e / kRing) & 1);
        } else if (warp == 2 || (warp == 3 && two)) {
            // ---------------- MMA issuer of tile t (the warp waits together, one lane issues)
            const int t = warp - 2;
            constexpr uint32_t id_s = tc::idesc_f16(kM, kN, false, false);
            constexpr uint32_t id_pv = tc::idesc_f16(kM, kD, false, true);
            constexpr uint32_t kHalf = kM * 8, kTileU = 2 * kHalf;   // 16-byte units of a 64-wide block, of a tile
            const uint64_t qd = tc::sdesc_sw128(smem_addr(s.q[t][0]), 16, 1024);
            const uint64_t kd = tc::sdesc_sw128(smem_addr(s.kv[0][0]), 16, 1024);
            const uint64_t vd = tc::sdesc_sw128(smem_addr(s.kv[0][0]), 2 * kN * 64, 1024);
            const uint32_t ts = tmem + kColS + t * kN, to = tmem + kColO + t * kD;
            auto full = [&](int e) { return wait_warp(s, &s.full[e % kRing], (e / kRing) & 1); };
            auto issue_s = [&](int j, uint32_t id) {
                const uint64_t b = kd + (uint32_t)(2 * j) % kRing * kTileU;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t o = (kk >> 2) * kHalf + (kk & 3) * 2;
                    tc::mma_ss(ts, qd + o, b + o, id, kk > 0);
                }
                tc::commit(&s.s_full[t]);
            };
            bool ok = wait_warp(s, &s.q_full, 0) && full(0);
            tc::fence_after_sync();
            if (ok && tc::elect_one()) {
                issue_s(0, few ? tc::idesc_f16(kM, kFew, false, false) : id_s);
                tc::commit(&s.done[0]);
            }
            for (int j = 0; ok && j < blk.n; ++j) {
                const bool next = j + 1 < blk.n;
                ok = full(2 * j + 1) && (!next || full(2 * j + 2)) && wait_warp(s, &s.p_full[t], j & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    const uint64_t b = vd + (uint32_t)(2 * j + 1) % kRing * kTileU;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < kFew / 16 || !few || j > 0)
                            tc::mma_ts(to, ts + kk * 8, b + kk * 128, id_pv, (j > 0) || (kk > 0));
                    if (next) issue_s(j + 1, id_s);
                    else tc::commit(&s.o_done[t]);
                    tc::commit(&s.done[(j + 1) & 1]);
                }
                __syncwarp();
            }
            // every MMA issued here has finished with shared and tensor memory before the CTA frees them
            if (tc::elect_one()) tc::commit(&s.drain[t]);
            __syncwarp();
            mbar_wait(&s.drain[t], 0);
        }
        __syncwarp();
    } else if (warp < 8 || two) {
        // ---------------- softmax warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
        const int t = warp >= 8;
        const Tile ti = t ? t1 : t0;
        const int r = 32 * (warp & 3) + lane;
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lane_off + kColS + t * kN, to = tmem + lane_off + kColO + t * kD;
        const int p = ti.p0 + r;   // this row's position
        const float sc = a.scale_log2;
        float m_ref = kNone;
        unsigned long long l2a = 0ull, l2b = 0ull;
        bool ok = true;
        if (few) {   // the sinks: as a block below, with kFew columns and a mask that is the same for every row
            ok = wait_warp(s, &s.s_full[t], 0);
            tc::fence_after_sync();
            uint32_t x[kFew], ph[kFew / 2];
            tc::tmem_ld32(ts, x);
            tc::wait_ld();
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < kFew; ++i) {
                if (i >= a.n_sink) x[i] = __float_as_uint(-INFINITY);
                mx = fmaxf(mx, __uint_as_float(x[i]));
            }
            m_ref = fmaxf(m_ref, mx * sc);
#pragma unroll
            for (int i = 0; i < kFew / 2; ++i) {
                const float p0 = ex2(fmaf(__uint_as_float(x[2 * i]), sc, -m_ref));
                const float p1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), sc, -m_ref));
                ph[i] = pack_half2(p0, p1);
                l2a = fadd2(l2a, f2pack(p0, p1));
            }
            tc::tmem_st16(ts, ph);
            tc::wait_st();
            tc::fence_before_sync();
            if (ok) tc::arrive_warp(&s.p_full[t]);
        }
        for (int j = few; ok && j < blk.n; ++j) {
            const int k0 = blk.at(j) * kN;
            // every row sees the whole block: no key after the first row's, all in the last row's window or sinks
            const bool whole = k0 + kN - 1 <= ti.p0 && (k0 >= ti.p1 - (a.window - 1) || k0 + kN <= a.n_sink);
            ok = wait_warp(s, &s.s_full[t], j & 1);
            if (!ok) break;
            tc::fence_after_sync();
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tc::tmem_ld32(ts + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&x[32 * c]));
            tc::wait_ld();
            if (!whole) {
                const int hi = p + 1 - k0, lo = p - (a.window - 1) - k0, sk = min(a.n_sink - k0, hi);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t seen = bits(lo - 32 * c, hi - 32 * c) | bits(0, sk - 32 * c);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(seen >> i & 1)) x[32 * c + i] = __float_as_uint(-INFINITY);
                }
            }
            float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
            for (int c = 0; c < 128; c += 8) {
                mx0 = max3(mx0, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                mx1 = max3(mx1, __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]));
                mx2 = max3(mx2, __uint_as_float(x[c + 4]), __uint_as_float(x[c + 5]));
                mx3 = max3(mx3, __uint_as_float(x[c + 6]), __uint_as_float(x[c + 7]));
            }
            const float mxs = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sc;
            float alpha = 1.f;
            const bool grow = mxs > m_ref + kLazy;
            if (grow) {
                alpha = ex2(m_ref - mxs);
                m_ref = mxs;
                const unsigned long long al2 = f2pack(alpha, alpha);
                l2a = fmul2(l2a, al2);
                l2b = fmul2(l2b, al2);
            }
            const unsigned long long sc2 = f2pack(sc, sc), nm2 = f2pack(-m_ref, -m_ref);
            uint32_t ph[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) {
                float e0, e1;
                f2unpack(ffma2(f2pack(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])), sc2, nm2), e0, e1);
                const float p0 = ex2(e0), p1 = ex2(e1);
                ph[c] = pack_half2(p0, p1);
                if (c & 1) l2b = fadd2(l2b, f2pack(p0, p1));
                else l2a = fadd2(l2a, f2pack(p0, p1));
            }
            tc::tmem_st32(ts, *reinterpret_cast<uint32_t(*)[32]>(&ph[0]));
            tc::tmem_st32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&ph[32]));
            if (j > 0 && __any_sync(0xffffffffu, grow)) {   // O holds every block before j (see above)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32(to + 32 * c, o);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tc::tmem_st32(to + 32 * c, o);
                }
            }
            tc::wait_st();
            tc::fence_before_sync();
            tc::arrive_warp(&s.p_full[t]);
        }
        // ---------------- epilogue: O / l -> fp16 -> swizzled smem (the Q tile) -> TMA store
        if (ok) ok = wait_warp(s, &s.o_done[t], 0);
        if (ok) {
            tc::fence_after_sync();
            unsigned char *qbytes = reinterpret_cast<unsigned char *>(s.q[t]);
            float la, lb;
            f2unpack(fadd2(l2a, l2b), la, lb);
            const float l = la + lb, inv = 1.f / l;
            uint32_t bad = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tc::tmem_ld32(to + 32 * c, o);
                tc::wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u) {   // 16-byte chunk: d = 32c + 8u .. +7
                    const int d = 32 * c + 8 * u;
                    const int kb = d >> 6, ch = (d & 63) >> 3;
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // exponent 31 carries into bit 15 of each half
                        w[i] = pack_half2(__uint_as_float(o[8 * u + 2 * i]) * inv, __uint_as_float(o[8 * u + 2 * i + 1]) * inv);
                        bad |= (w[i] & 0x7C007C00u) + 0x04000400u;
                    }
                    *reinterpret_cast<uint4 *>(qbytes + kb * (kM * 128) + r * 128 + ((ch ^ (r & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            // (weights that are NaN themselves, or none at all, give NaN whatever the values are)
            uint32_t again = __ballot_sync(0xffffffffu, (bad & 0x80008000u) && l > 0.f && l < INFINITY && ti.q0 + r < a.Tq);
            __syncwarp();   // the rows' lanes have written them
            if (again)
                again = explain_rows(a, blk, few, unit, ti.p0 + 32 * (warp & 3), again, qbytes + 32 * (warp & 3) * 128, lane);
            for (; again; again &= again - 1) {
                const int ra = 32 * (warp & 3) + __ffs(again) - 1;
                slow_row(a, ((size_t)b * a.Hq + ti.h) * a.Tq + ti.q0 + ra, unit, ti.p0 + ra, qbytes + ra * 128, ra & 7, lane);
            }
            tc::fence_proxy_async_smem();
        }
        asm volatile("bar.sync %0, 128;\n" ::"r"(1 + t) : "memory");
        if (ok && (warp & 3) == 0 && lane == 0) {
            tc::tma_store_3d(&map_o, s.q[t][0], 0, ti.q0, b * a.Hq + ti.h);
            tc::tma_store_3d(&map_o, s.q[t][1], 64, ti.q0, b * a.Hq + ti.h);
            tc::bulk_commit_group();
            tc::bulk_wait_read();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
    if (tid < (two ? 2 : 1)) a.status[unit * a.ntile + first + tid] = s.abort ? 1u : 0u;
}

std::mutex g_attr_mu;
bool g_attr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};

long long tiles_of(int Hq, int Hkv, int Tq) { return ((long long)Tq + kM - 1) / kM * (Hq / Hkv); }

// Query tiles of a CTA: two share every K / V block they read and hide each
// other's softmax (8192 tokens, window 4096: 430 us); one while there are SMs for
// all of them, as a tile alone is done sooner (512 tokens, window 128, 4 heads:
// 18.4 us with CTAs of two, 12.3 with one; 8.5 now).
int tiles_per_cta(int B, int Hq, int Hkv, int Tq, int sms) {
    return (long long)B * Hkv * tiles_of(Hq, Hkv, Tq) <= sms ? 1 : 2;
}

}  // namespace

// Workspace: a status word a query tile.
size_t window_prefill_status_words(int B, int Hq, int Hkv, int Tq) {
    return (size_t)B * Hkv * (size_t)tiles_of(Hq, Hkv, Tq);
}
size_t window_prefill_workspace_bytes(int B, int Hq, int Hkv, int Tq) {
    return (window_prefill_status_words(B, Hq, Hkv, Tq) * 4 + 255) / 256 * 256;
}

int window_prefill_launch(const uint16_t *q, const uint16_t *k, const uint16_t *v, int B, int Hq, int Hkv, int Tq,
                          int Tk, int window, int n_sink, float sm_scale, uint16_t *o, void *ws, cudaStream_t stream) {
    CUtensorMap mq, mk, mv, mo;
    int rc;
    if ((rc = make_row_map(&mq, q, Tq, B * Hq, "window_prefill: q")) ||
        (rc = make_row_map(&mk, k, Tk, B * Hkv, "window_prefill: k")) ||
        (rc = make_row_map(&mv, v, Tk, B * Hkv, "window_prefill: v")) ||
        (rc = make_row_map(&mo, o, Tq, B * Hq, "window_prefill: o")))
        return rc;
    Args a;
    a.q = q; a.k = k; a.v = v;
    a.status = static_cast<unsigned *>(ws);
    a.Hq = Hq; a.Hkv = Hkv; a.Tq = Tq; a.Tk = Tk;
    a.window = window < Tk ? window : Tk;   // the same keys, and no overflow in the kernel's differences
    a.n_sink = n_sink < Tk ? n_sink : Tk;
    a.units = B * Hkv;
    a.ntile = (Tq + kM - 1) / kM * (Hq / Hkv);
    a.scale_log2 = sm_scale * kLog2e;
    const size_t smem = sizeof(Smem) + 1024;
    const int dev = current_device();
    if (dev < 0) return fail(MINIKV_ERR_CUDA, "window_prefill: no current CUDA device");
    {
        std::lock_guard<std::mutex> lk(g_attr_mu);
        if (!g_attr[dev]) {
            if (cudaFuncSetAttribute(window_fa_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
                cudaSuccess)
                return check_launch("window_prefill: attribute");
            int sms = 148;
            if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) sms = 148;
            g_sms[dev] = sms;
            g_attr[dev] = true;
        }
        a.per = tiles_per_cta(B, Hq, Hkv, Tq, g_sms[dev]);
    }
    a.ncta = (a.ntile + a.per - 1) / a.per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.units * a.ncta));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, window_fa_kernel, mq, mk, mv, mo, a);
    return check_launch("window_prefill");
}

}  // namespace minikv

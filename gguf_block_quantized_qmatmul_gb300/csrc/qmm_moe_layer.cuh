// qmm_moe_layer.cuh -- a whole mixture-of-experts layer for a few tokens in two
// launches.
//
// Mathematics: that of the four calls that it stands for.  l = x R^T in f32;
// the routing of qmm_moe_route.cu; h = silu(x Wg^T) (x Wu^T) of each token's
// experts; y = sum_j p_j (h_j Wd^T).  The products are the row kernel's
// (qmm_q4g_rows.cuh): codes less their zero point are exact operands of f16 or
// bf16 warp MMAs, group sums are scaled in f32, an f32 activation is three bf16
// pieces.  h is two pieces of a 16-bit type between the two (f32: as it is): rounded to one, its error was as large as the result's
// own rounding (2.9e-4 for 2.1e-4 in f16).  The pieces are columns that an
// MMA has anyway.
//
// A decode step's layer reads a few MB of weights, 100 KB an SM, so what stands
// between the products is what costs.  The first launch forms the logits (a
// block per expert).  In the second every block routes all tokens for itself
// (a warp a token, no exchange), then takes shares of the work by tickets: first
// shares of the experts' first products, then of the second ones, which wait
// until all of the first are reported, and, unless an item is a token, of the
// tokens' sums.  A ticket's holder runs already when it waits, and what it waits
// for are shares with lower tickets, whose holders do not wait for it: however
// few blocks are on the GPU at a time, the layer ends.  The tokens are staged
// beside the first launch, and the second products' weights are on their way
// before their block waits.
//
// A share is row blocks of items, end to end.  An item is an expert with up to 8
// (h: 4, f32: 2) of its tokens, whose pieces are the MMA's columns; for up to 4 tokens the second
// products' items are tokens, whose experts' segments are one long row.  A share's
// segments of 16 x 128 weights are dealt to the block's warps in equal
// contiguous runs, wherever row blocks end, so that no warp has more to do than
// another; each streams its own through a ring of asynchronous copies, and no
// warp waits for another until the end, where the parts of row blocks that were
// cut are added in shared memory, in the order of K.  (Whole row blocks to groups of
// warps, as the row kernel deals them: 16 tokens of 64 experts 31 us for the
// first products, and 8 more in blocks whose share held two experts.)
//
// Measured (2048 -> 2 x 1024 -> 2048, 8 of 64 experts, us): 1 token in bf16 20 (logits 5, routing 3, products 6 and
// 4, the wait between them 2), 4 35, 8 46, 16 in f16 58 (28 at the peak; products 24 and 12, 5.6 TB/s), 32 68.
//
// Waits are bounded: one that gives up raises the error word and its block ends.
#pragma once

#include <type_traits>

#include "qmm_moe_route.cuh"
#include "qmm_q4g_rows.cuh"

namespace qmm {

constexpr int kMoeWarps = 16, kMoeThreads = kMoeWarps * 32;
constexpr int kMoeDepth = 6;     // segments in a warp's ring
constexpr int kMoeItems = 8;     // items of a share that are staged together, at most
constexpr int kMoeStatic = 1024; // the kernel's static arrays, rounded up
constexpr int kMoePart = kMoeWarps * 2 * 512;  // bytes of the parts of row blocks

struct MoeParams {
    RouteParams route;   // c.ids, c.weights: for the caller, or NULL
    QgWeights up, down;
    const void* x;
    long long ldx;
    int xt;
    void* h;             // [T top_k][F] f32, or [T top_k][2][F] pieces of the activations' type
    float* part;         // [T top_k][N]: the experts' second products, unless items are tokens
    void* y;
    unsigned* counters;  // [0] tickets, [1] shares of the first products done, [2] of the second
    unsigned* err;
    int epl16;           // experts per lane in the routing: 16, or 4
    int up_log2, down_log2;  // tokens per item, at most
    int up_cols, down_cols;  // and how many have room
    int whole, up_items, down_items;
    int off_zero, off_part, off_ring, off_route;
    int stall;
};

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void add_release(unsigned* p) { asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory"); }

// Waits until *p is n; called by one thread.
static __device__ __noinline__ bool moe_wait(const unsigned* p, unsigned n, unsigned* err) {
    const long long t0 = clock64();
    long long lim = 0;
    while (ld_acquire(p) != n) {
        const long long dt = clock64() - t0;
        if (dt <= kWaitLimitCheck) continue;
        if (lim == 0) lim = wait_limit(err);
        if (dt > lim) {
            atomicOr(err, ERR_TIMEOUT);
            return false;
        }
        __nanosleep(100);
    }
    return true;
}

// An item of an expert: its tokens' slots are order[first .. first + n).  In one word: 512 experts, 1024 slots.
struct MoeItem {
    uint32_t v;
    __device__ __forceinline__ int expert() const { return (int)(v & 511u); }
    __device__ __forceinline__ int first() const { return (int)(v >> 9 & 1023u); }
    __device__ __forceinline__ int n() const { return (int)(v >> 19); }
};
// The routing, in shared memory.
struct MoeShared {
    const int* ids;         // [T][top_k]
    const float* weights;
    const int* order;       // slots by expert
    const int* token;       // and their tokens
    const MoeItem* items;
    int T, k;
};

// Where a share's segments are: run r (KS segments of one row block of one expert) of a batch that
// begins with row block rb0 of item i0.
template <bool TOKEN>
struct MoeRun {
    int item, rb, j;  // TOKEN: choice j of token `item`
    __device__ __forceinline__ MoeRun(const MoeShared& sh, int i0, int rb0, int RB, int r) {
        int u = r;
        j = 0;
        if (TOKEN) {
            u = r / sh.k;
            j = r - u * sh.k;
        }
        const int b = rb0 + u;
        const int di = b / RB;
        item = i0 + di;
        rb = b - di * RB;
    }
    // true: a row block is complete
    __device__ __forceinline__ bool next(const MoeShared& sh, int RB) {
        if (TOKEN && ++j < sh.k) return false;
        j = 0;
        if (++rb == RB) {
            rb = 0;
            ++item;
        }
        return true;
    }
    __device__ __forceinline__ int expert(const MoeShared& sh) const { return TOKEN ? sh.ids[item * sh.k + j] : sh.items[item].expert(); }
};

// Stages nh x rows quads of 32 values: block h of row r is `left` values (none: <= 0) from element
// src(r, h, left) of x on, and goes to 64 bytes at h * rows + r.  S32: x is f32, three bf16 pieces of 64 bytes
// by truncation (exact, no overflow).  B loads a thread are in flight.
template <int B, bool S32, class Src>
__device__ __forceinline__ void moe_stage(uint8_t* sm, const void* x, int nh, int rows, Src src, int tid) {
    constexpr int NP = S32 ? 3 : 1;
    const int n = nh * rows * 4;
    for (int i0 = 0; i0 < n; i0 += B * kMoeThreads) {
        uint4 u[B][S32 ? 2 : 1];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * kMoeThreads + tid, quad = i >> 2, h = quad / rows;
#pragma unroll
            for (int q = 0; q < (S32 ? 2 : 1); ++q) u[b][q] = make_uint4(0u, 0u, 0u, 0u);
            if (i < n) {
                int left;
                const long long at = src(quad - h * rows, h, left) + 8 * (i & 3);
                if (8 * (i & 3) < left)
#pragma unroll
                    for (int q = 0; q < (S32 ? 2 : 1); ++q) u[b][q] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + at * (S32 ? 4 : 2)) + q);  // past L1, which may hold an earlier x or h
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int i = i0 + b * kMoeThreads + tid, j = i & 3;
            if (i - (tid & 31) >= n) break;  // the whole warp is done
            uint8_t* to = sm + (long long)(i >> 2) * (NP * 64) + j * 16;
            if constexpr (S32) {
                float f[8] = {__uint_as_float(u[b][0].x), __uint_as_float(u[b][0].y), __uint_as_float(u[b][0].z), __uint_as_float(u[b][0].w),
                              __uint_as_float(u[b][1].x), __uint_as_float(u[b][1].y), __uint_as_float(u[b][1].z), __uint_as_float(u[b][1].w)};
#pragma unroll
                for (int pc = 0; pc < NP; ++pc) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        // the rest is exact; an infinity or NaN has none
                        const uint32_t lo = __float_as_uint(f[e]) & 0xffff0000u, hi = __float_as_uint(f[e + 1]) & 0xffff0000u;
                        w[e >> 1] = hi | lo >> 16;
                        f[e] = (lo & 0x7f800000u) == 0x7f800000u ? 0.0f : f[e] - __uint_as_float(lo);
                        f[e + 1] = (hi & 0x7f800000u) == 0x7f800000u ? 0.0f : f[e + 1] - __uint_as_float(hi);
                    }
                    const uint4 q = qg_quad_transpose(w[0], w[1], w[2], w[3], j);
                    if (i < n) *reinterpret_cast<uint4*>(to + pc * 64) = q;
                }
            } else {
                const uint4 q = qg_quad_transpose(u[b][0].x, u[b][0].y, u[b][0].z, u[b][0].w, j);
                if (i < n) *reinterpret_cast<uint4*>(to) = q;
            }
        }
    }
}

// Row blocks w0 .. w1 of one product's items.  UP: the first product, x to h; else the second, h to part
// (TOKEN: y).  wait() (false: give up) comes before the activations are read.
template <bool BF, bool F32, int NG, bool UP, bool TOKEN, class Wait>
__device__ __forceinline__ bool moe_share(const MoeParams& p, const QgWeights& w, uint8_t* sm, const MoeShared& sh, int w0, int w1, Wait wait) {
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
    constexpr int seg_bytes = qg_seg_bytes(NG), segk = 128 / NG, np = F32 ? 3 : UP ? 1 : 2, kFlight = F32 ? 2 : 4;
    const int KS = w.KS, RB = w.RB, kk = TOKEN ? sh.k : 1;  // runs per row block
    const long long rb_bytes = (long long)KS * seg_bytes;
    uint8_t* ring = sm + p.off_ring + warp * (kMoeDepth * seg_bytes);
    float4* parts = reinterpret_cast<float4*>(sm + p.off_part);  // [warp][2][32]: a row block's part that does not reach its end: 1; that does: 0
    const uint32_t magic = opaque(kQgMagic<BF>);
    const bool whole = UP && p.whole;
    // a staged item: [32 K][columns] of 64 bytes
    const int item_bytes = (TOKEN ? sh.k : UP ? p.up_cols : p.down_cols) * np * KS * 256;
    const int batch = UP ? (whole ? kMoeItems * 16 : p.up_items) : p.down_items;
    bool ok = true;
    for (int b0 = w0; b0 < w1;) {
        const int i0 = b0 / RB, rb0 = b0 - i0 * RB;
        const int b1 = min(w1, (i0 + batch) * RB);
        // this warp's segments of the batch
        const int units = b1 - b0, per = kk * KS, total = units * per;
        const int s0 = (int)((long long)warp * total / kMoeWarps), s1 = (int)((long long)(warp + 1) * total / kMoeWarps);
        int lleft = s1 - s0, lrem = KS - s0 % KS, ls = 0;
        MoeRun<TOKEN> lr(sh, i0, rb0, RB, s0 / KS);
        const uint8_t* lp = nullptr;
        auto place = [&](int seg) { lp = w.data + (long long)lr.expert(sh) * w.expert_stride + lr.rb * rb_bytes + seg * seg_bytes + lane * 16; };
        if (lleft > 0) place(KS - lrem);
        const uint32_t to = smem_u32(ring) + lane * 16;
        auto load = [&]() {  // a group of copies, empty past the end, so that the groups' count is the ring's
            if (lleft > 0) {
                const uint32_t d = to + ls * seg_bytes;
                cp_async16(d, lp);
                cp_async16(d + kQgTile, lp + kQgTile);
                if (lane < 4 * NG) cp_async16(d + 2 * kQgTile, lp + 2 * kQgTile);
                lp += seg_bytes;
                --lleft;
                if (--lrem == 0 && lleft > 0) {
                    lrem = KS;
                    lr.next(sh, RB);
                    place(0);
                }
            }
            ls = ls + 1 == kMoeDepth ? 0 : ls + 1;
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kMoeDepth - 1; ++i) load();
        if (!(ok = wait())) break;
        if (!whole) {
            const int i1 = (b1 - 1) / RB;
            for (int it = i0; it <= i1; ++it) {
                uint8_t* area = sm + (it - i0) * item_bytes;
                constexpr int pieces = !UP && !F32 ? 2 : 1;  // rows of an activation row
                if (TOKEN) {  // its choices' rows end to end
                    const int per_row = KS * 4;
                    moe_stage<kFlight, F32>(area, p.h, sh.k * per_row, pieces, [&](int pc, int h, int& left) {
                        const int j = h / per_row, k32 = 32 * (h - j * per_row);
                        left = w.K - k32;
                        return (((long long)it * sh.k + j) * pieces + pc) * w.K + k32;
                    }, tid);
                } else {
                    const MoeItem m = sh.items[it];
                    moe_stage<kFlight, F32>(area, UP ? p.x : p.h, KS * 4, m.n() * pieces, [&](int r, int h, int& left) {
                        left = w.K - 32 * h;
                        if (UP) return sh.token[m.first() + r] * p.ldx + 32 * h;
                        return ((long long)sh.order[m.first() + r / pieces] * pieces + r % pieces) * w.K + 32 * h;
                    }, tid);
                }
            }
            __syncthreads();
        }

        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        // This lane's activations: at xo, xq bytes from 32 K to the next (0: it has no column).  Column g is
        // token g of the item, or piece g % 2 (3 pieces: g % 4) of token g / 2 (g / 4).
        int xo = 0, xq = 0;
        float wt = 1.0f;
        auto columns = [&](const MoeRun<TOKEN>& r, int seg) {
            const int n = TOKEN ? 1 : sh.items[r.item].n(), c = np == 3 ? g >> 2 : np == 2 ? g >> 1 : g, pc = np == 3 ? g & 3 : np == 2 ? g & 1 : 0;
            if (c < n && pc < np) {
                int base, ncol;
                if (whole) {
                    ncol = sh.T * np;
                    base = (sh.token[sh.items[r.item].first() + c] * np + pc) * 64;
                } else {
                    ncol = n * np;
                    base = (r.item - i0) * item_bytes + (c * np + pc) * 64 + (TOKEN ? r.j * KS * 4 * ncol * 64 : 0);
                }
                xq = ncol * 64;
                xo = base + seg * 4 * xq + t * 16;
            } else {
                xq = 0;
                xo = p.off_zero;
            }
            if (TOKEN) wt = sh.weights[r.item * sh.k + r.j];
        };
        // a row block's 16 x 8 sums to their place
        auto put = [&](float v[4], int item, int rb) {
            if (np > 1) {  // pieces 0, 1 are one lane's, piece 2 its neighbour's
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    v[i] += v[i + 1];
                    if (np == 3) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 1);
                }
            }
            constexpr float unit = BF ? 1.0f / kQgCodeUnit : 1.0f;
            const MoeItem it = TOKEN ? MoeItem{0u} : sh.items[item];
            const int n = TOKEN ? 1 : it.n();
#pragma unroll
            for (int i = 0; i < (np > 1 ? 1 : 2); ++i) {
                const int c = np == 3 ? t >> 1 : np == 2 ? t : 2 * t + i;
                if (c >= n || (np == 3 && (t & 1))) continue;
                const float lo = v[i] * unit, hi = v[i + 2] * unit;
                if (UP) {
                    const int f = rb * 8 + g, F = w.N / 2;
                    if (f >= F) continue;
                    const long long slot = sh.order[it.first() + c];
                    const float v = swiglu(lo, hi);
                    if constexpr (F32) {
                        static_cast<float*>(p.h)[slot * F + f] = v;
                    } else {
                        using H = typename std::conditional<BF, __nv_bfloat16, __half>::type;
                        H* to = static_cast<H*>(p.h) + slot * 2 * F + f;
                        const H one = to_type<H>(v);
                        const float rest = v - (float)one;
                        to[0] = one;
                        to[F] = to_type<H>(fabsf((float)one) < INFINITY ? rest : 0.0f);  // an infinity or NaN has none
                    }
                } else {
                    const int row = rb * 16 + g;
                    if (TOKEN) {
                        if (row < w.N) x_store(p.y, p.xt, (long long)item * w.N + row, lo);
                        if (row + 8 < w.N) x_store(p.y, p.xt, (long long)item * w.N + row + 8, hi);
                    } else {
                        float* out = p.part + (long long)sh.order[it.first() + c] * w.N;
                        if (row < w.N) out[row] = lo;
                        if (row + 8 < w.N) out[row + 8] = hi;
                    }
                }
            }
        };
        // The row block that this warp completes but did not begin, which it puts in its place at the end.
        int cut = -1, cut_item = 0, cut_rb = 0;
        MoeRun<TOKEN> r(sh, i0, rb0, RB, s0 / KS);
        int cs = 0, seg = s0 % KS;  // ring place, segment in the run
        int first = s0 - s0 % per, begin = s0;  // where the row block and this warp's part of it begin
        for (int i = s0; i < s1; seg = 0) {
            const int end = min(s1, i - seg + KS);
            const bool run_done = end == i - seg + KS;
            columns(r, seg);
            for (; i < end; ++i) {
                cp_async_wait<kMoeDepth - 2>();
                __syncwarp();  // every lane's copies of this segment have landed, and the last one has been read
                load();
                const uint8_t* sp = ring + cs * seg_bytes;
                cs = cs + 1 == kMoeDepth ? 0 : cs + 1;
                const uint4 c0 = reinterpret_cast<const uint4*>(sp)[lane], c1 = reinterpret_cast<const uint4*>(sp + kQgTile)[lane];
                uint32_t sw[2 * NG];
                const uint8_t* sq = sp + 2 * kQgTile + g * (8 * NG);
                if (NG == 1) {
                    const uint2 u = *reinterpret_cast<const uint2*>(sq);
                    sw[0] = u.x;
                    sw[1] = u.y;
                } else {
#pragma unroll
                    for (int q = 0; q < NG / 2; ++q) {
                        const uint4 u = reinterpret_cast<const uint4*>(sq)[q];
                        sw[4 * q] = u.x;
                        sw[4 * q + 1] = u.y;
                        sw[4 * q + 2] = u.z;
                        sw[4 * q + 3] = u.w;
                    }
                }
                float gr[4];
                uint32_t zl = 0, zh = 0;
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {  // 32 K a step
                    const int gi = q4 * 32 / segk;
                    const uint32_t sw0 = sw[2 * gi], sw1 = sw[2 * gi + 1];
                    const bool start = q4 * 32 % segk == 0;
                    if (start) {
                        zl = qg_zero<BF>(sw0, false);
                        zh = qg_zero<BF>(sw1, true);
                    }
                    const uint4 cw = q4 < 2 ? c0 : c1;
                    uint32_t a0[4], a1[4];
                    qg_codes<BF>(q4 & 1 ? cw.z : cw.x, magic, zl, zh, a0);
                    qg_codes<BF>(q4 & 1 ? cw.w : cw.y, magic, zl, zh, a1);
                    const uint4 xv = *reinterpret_cast<const uint4*>(sm + xo + q4 * xq);
                    if (start) qg_mma<BF, true>(gr, a0, xv.x, xv.y);
                    else qg_mma<BF, false>(gr, a0, xv.x, xv.y);
                    qg_mma<BF, false>(gr, a1, xv.z, xv.w);
                    if ((q4 + 1) * 32 % segk == 0) {  // the group's end
                        const float f0 = TOKEN ? qg_scale(sw0) * wt : qg_scale(sw0), f1 = TOKEN ? qg_scale(sw1) * wt : qg_scale(sw1);
                        acc[0] = fmaf(f0, gr[0], acc[0]);
                        acc[1] = fmaf(f0, gr[1], acc[1]);
                        acc[2] = fmaf(f1, gr[2], acc[2]);
                        acc[3] = fmaf(f1, gr[3], acc[3]);
                    }
                }
                xo += 4 * xq;
            }
            const int item = r.item, rb = r.rb;
            const bool done = run_done && r.next(sh, RB);
            if (!done && i < s1) continue;  // TOKEN: the next choice
            if (done && begin == first) {
                put(acc, item, rb);
            } else {
                parts[(warp * 2 + (done ? 0 : 1)) * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (done) {
                    cut = first;
                    cut_item = item;
                    cut_rb = rb;
                }
            }
            acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
            first = begin = i;
        }
        cp_async_wait<0>();
        __syncthreads();  // all parts are there, and the activations are no longer read
        if (cut >= 0) {
            int from = warp - 1;
            while ((int)((long long)from * total / kMoeWarps) > cut) --from;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int o = from; o <= warp; ++o) {
                if ((int)((long long)o * total / kMoeWarps) == (int)((long long)(o + 1) * total / kMoeWarps)) continue;  // no segments
                const float4 u = parts[(o * 2 + (o == warp ? 0 : 1)) * 32 + lane];
                v[0] += u.x;
                v[1] += u.y;
                v[2] += u.z;
                v[3] += u.w;
            }
            put(v, cut_item, cut_rb);
        }
        b0 = b1;
        if (b0 < w1) __syncthreads();  // the parts have been read
    }
    cp_async_wait<0>();
    return ok;
}

template <bool BF, bool F32, bool TOKEN>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_layer_kernel(const __grid_constant__ MoeParams p) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int s_ok, s_items[2];  // [1]: of the second products
    __shared__ unsigned s_ticket[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = p.route.c.T, E = p.route.c.E, k = p.route.c.top_k, S = T * k;
    int* ids = reinterpret_cast<int*>(sm + p.off_route);             // [S]
    float* weights = reinterpret_cast<float*>(ids + S);              // [S]
    int* order = reinterpret_cast<int*>(weights + S);                // [S]
    int* token = order + S;                                          // [S]
    MoeItem* items = reinterpret_cast<MoeItem*>(token + S);          // [S] of the first products
    MoeItem* items2 = items + S;                                     // [S] of the second
    using Sum = unsigned long long;
    Sum* before = reinterpret_cast<Sum*>(items2 + S);                // [E] slots, first and second items before an expert's
    uint32_t* mask = reinterpret_cast<uint32_t*>(before + E);        // [E] the tokens that chose an expert
    uint32_t* picks = reinterpret_cast<uint32_t*>(sm + p.off_ring);  // [warps][E], where the rings will be
    for (int e = tid; e < E; e += kMoeThreads) mask[e] = 0u;
    if (tid == 0) *reinterpret_cast<uint4*>(sm + p.off_zero) = make_uint4(0u, 0u, 0u, 0u);  // what lanes without a column read
    grid_dep_launch();
    // The first launch lets this one start only when what it depends on itself has completed, so the
    // tokens are there.
    if (p.whole)
        moe_stage<F32 ? 2 : 4, F32>(sm, p.x, p.up.KS * 4, T, [&](int r, int h, int& left) {
            left = p.up.K - 32 * h;
            return r * p.ldx + 32 * h;
        }, tid);
    grid_dep_wait();
    unsigned next = 0;  // thread 0: the next ticket
    if (tid == 0) next = atomicAdd(p.counters, 1u);
    __syncthreads();

    // ------------------------------ routing ------------------------------
    RouteParams rp = p.route;
    rp.c.ids = ids;
    rp.c.weights = weights;
    for (int t = warp; t < T; t += kMoeWarps) {
        const int id = p.epl16 ? route_token<16>(rp, t, picks + warp * E, lane) : route_token<4>(rp, t, picks + warp * E, lane);
        if (lane < k) atomicOr(&mask[id], 1u << t);
    }
    __syncthreads();
    if (warp == 0) {
        // Slots sorted by expert, by token within one: a count is a mask's population, a rank that of its
        // lower bits.  Slots and both products' items before each expert are one sum's thirds.
        const int per = (E + 31) / 32;
        auto count = [&](int n) { return (Sum)n | (Sum)((n + (1 << p.up_log2) - 1) >> p.up_log2) << 16 | (Sum)((n + (1 << p.down_log2) - 1) >> p.down_log2) << 32; };
        Sum mine = 0;
        for (int i = 0; i < per; ++i)
            if (lane * per + i < E) mine += count(__popc(mask[lane * per + i]));
        Sum pre = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum u = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += u;
        }
        if (lane == 31) {
            s_items[0] = (int)(pre >> 16 & 0xffffu);
            s_items[1] = (int)(pre >> 32);
        }
        pre -= mine;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e >= E) break;
            before[e] = pre;
            pre += count(__popc(mask[e]));
        }
    }
    __syncthreads();
    for (int s = tid; s < S; s += kMoeThreads) {
        const int t = s / k, e = ids[s], at = (int)(before[e] & 0xffffu) + __popc(mask[e] & ((1u << t) - 1u));
        order[at] = s;
        token[at] = t;
        if (blockIdx.x == 0 && p.route.c.ids) {
            p.route.c.ids[s] = e;
            p.route.c.weights[s] = weights[s];
        }
    }
    for (int e = tid; e < E; e += kMoeThreads) {
        const Sum pre = before[e];
        const int n = __popc(mask[e]), first = (int)(pre & 0xffffu);
        auto list = [&](MoeItem* to, int cols) {
            for (int c = 0; c < n; c += cols) *to++ = MoeItem{(uint32_t)e | (uint32_t)(first + c) << 9 | (uint32_t)min(cols, n - c) << 19};
        };
        list(items + (pre >> 16 & 0xffffu), 1 << p.up_log2);
        list(items2 + (pre >> 32), 1 << p.down_log2);
    }
    const MoeShared sh = {ids, weights, order, token, items, T, k}, sh2 = {ids, weights, order, token, items2, T, k};

    // ------------------------------ shares ------------------------------
    // The next ticket is drawn when a share begins and known to all when it ends, at one barrier.
    const unsigned G = gridDim.x, total = TOKEN ? 2 * G : 3 * G;
    if (tid == 0) s_ticket[0] = next;
    __syncthreads();
    for (int it = 0;; ++it) {
        const unsigned ticket = s_ticket[it & 1];
        if (ticket >= total) break;
        if (tid == 0) next = atomicAdd(p.counters, 1u);
        const unsigned phase = ticket / G, i = ticket - phase * G;
        // what others make: waited for by one thread
        bool waited = false;
        auto wait = [&](unsigned which) {
            if (waited) return true;
            waited = true;
            if (tid == 0) s_ok = moe_wait(p.counters + which, G, p.err);
            __syncthreads();
            return s_ok != 0;
        };
        bool ok;
        if (phase == 0) {
            const unsigned work = (unsigned)s_items[0] * p.up.RB;  // times the blocks: below 2^32, as planned
            const int w0 = (int)(i * work / G), w1 = (int)((i + 1) * work / G);
            auto no = [] { return true; };
            if (p.up.ng == 1) ok = moe_share<BF, F32, 1, true, false>(p, p.up, sm, sh, w0, w1, no);
            else if (p.up.ng == 2) ok = moe_share<BF, F32, 2, true, false>(p, p.up, sm, sh, w0, w1, no);
            else ok = moe_share<BF, F32, 4, true, false>(p, p.up, sm, sh, w0, w1, no);
        } else if (phase == 1) {
            const unsigned work = (unsigned)(TOKEN ? T : s_items[1]) * p.down.RB;
            const int w0 = (int)(i * work / G), w1 = (int)((i + 1) * work / G);
            auto first = [&] { return wait(1u); };
            if (p.down.ng == 1) ok = moe_share<BF, F32, 1, false, TOKEN>(p, p.down, sm, sh2, w0, w1, first);
            else if (p.down.ng == 2) ok = moe_share<BF, F32, 2, false, TOKEN>(p, p.down, sm, sh2, w0, w1, first);
            else ok = moe_share<BF, F32, 4, false, TOKEN>(p, p.down, sm, sh2, w0, w1, first);
        } else {
            // a token's second products, in the order of its choices
            if ((ok = wait(2u))) {
                const int N = p.down.N;
                const long long n = (long long)T * N, o1 = (long long)(i + 1) * n / G;
                for (long long o = (long long)i * n / G + tid; o < o1; o += kMoeThreads) {
                    const int t = (int)(o / N), col = (int)(o - (long long)t * N);
                    float v = 0.0f;
#pragma unroll 8
                    for (int j = 0; j < k; ++j) v = fmaf(weights[t * k + j], __ldcg(p.part + (long long)(t * k + j) * N + col), v);
                    x_store(p.y, p.xt, o, v);
                }
            }
        }
        if (!ok) break;
        if (tid == 0) s_ticket[(it + 1) & 1] = next;
        __syncthreads();  // every thread's results are written, and what the share kept in shared memory is no longer read
        // by the last warp's first thread: its fence takes a while, and only its own warp's next loads wait for it
        if (tid == kMoeThreads - 32 && phase < (TOKEN ? 1u : 2u) && !(p.stall && ticket == 0)) add_release(p.counters + 1 + phase);
    }
}

template <bool BF, bool F32, bool TOKEN>
cudaError_t moe_layer_go(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s) {
    static unsigned long long done = 0;
    auto* k = moe_layer_kernel<BF, F32, TOKEN>;
    const cudaError_t e = ensure_smem(k, smem_max - kMoeStatic, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, (unsigned)pl.blocks, kMoeThreads, pl.smem, s, p);
}

}  // namespace qmm

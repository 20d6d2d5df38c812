// qmm_moe_layer.cu -- host side of the mixture-of-experts layer for a few
// tokens (qmm_moe_layer.cuh), and the router's product.
#include "qmm_moe_layer.cuh"

namespace qmm {

cudaError_t launch_moe_layer_f16(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s);
cudaError_t launch_moe_layer_bf16(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s);
cudaError_t launch_moe_layer_f32(const MoePlan& pl, const MoeParams& p, int smem_max, cudaStream_t s);

namespace {

__device__ __forceinline__ void router_load8(const void* row, int type, int k, float f[8]) {
    if (type == X_F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + k);
        const float4 b = *(reinterpret_cast<const float4*>(static_cast<const float*>(row) + k) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        return;
    }
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + k);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (type == X_F16) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

// Logits of four tokens for one expert a block: f32 products and sums in a fixed order.  Bound by
// latency: the router's row is asked into L2 before what this grid depends on has completed, and read after it, as
// the router is a caller's floats, which that may write; with it the tokens' values, all at once; one reduction.
// (A block for all tokens of an expert: 9 us for 16.)
// The first block clears the next launch's counters.
constexpr int kRouterTokens = 4;
__global__ void __launch_bounds__(256) moe_router_kernel(const void* x, int xt, long long ldx, int T, int K, const void* router, int rt, float* logits, int ldl,
                                                         unsigned* counters) {
    __shared__ float red[kRouterTokens][8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
    const uint8_t* w = static_cast<const uint8_t*>(router) + (long long)e * K * x_size(rt);
    for (int k = 8 * tid; k < K; k += 2048) asm volatile("prefetch.global.L2 [%0];" ::"l"(w + (long long)k * x_size(rt)));
    // the next launch reads x before this one has completed: it may start only now that x is there
    grid_dep_wait();
    grid_dep_launch();
    float f[8];
    if (8 * tid < K) router_load8(w, rt, 8 * tid, f);
    if (e == 0 && t0 == 0 && tid < 4) counters[tid] = 0u;
    float acc[kRouterTokens];
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) acc[t] = 0.0f;
    for (int k = 8 * tid; k < K;) {
        float v[kRouterTokens][8];
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t)  // past the last token: that one again
            router_load8(static_cast<const uint8_t*>(x) + min(t0 + t, T - 1) * ldx * x_size(xt), xt, k, v[t]);
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[t] = fmaf(f[i], v[t][i], acc[t]);
        if ((k += 2048) < K) router_load8(w, rt, k, f);
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
#pragma unroll
        for (int o = 16; o; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        if (lane == 0) red[t][warp] = acc[t];
    }
    __syncthreads();
    if (tid < kRouterTokens && t0 + tid < T) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += red[tid][i];
        logits[(long long)(t0 + tid) * ldl + e] = v;
    }
}

}  // namespace

MoePlan plan_moe_layer(const MoeCall& c, int sms, int smem_max) {
    MoePlan pl;
    const int T = c.T, k = c.route.top_k, S = T * k, E = c.up.E, np = c.xt == X_F32 ? 3 : 1;
    if (T < 1 || T > kMoeMaxTokens || E > kQgRowMaxE) return pl;
    // shared memory: activations, a zero, the parts of row blocks, the rings, the routing
    const int seg = qg_seg_bytes(c.up.ng > c.down.ng ? c.up.ng : c.down.ng), ring = kMoeWarps * kMoeDepth * seg;
    const int route = round_up((6 * S + 3 * E) * 4, 16);
    const int room = smem_max - kMoeStatic - 1024 - 16 - kMoePart - ring - route;
    const long long up_row = (long long)np * c.up.KS * 256, down_row = (long long)(np == 3 ? 3 : 2) * c.down.KS * 256;  // a token's, a slot's staged bytes
    // A token's second products end to end while few tokens share an expert: no partial sums to add later.  (1, 2, 4
    // tokens of 64 experts: 20.4, 25.6, 35.9 us; by expert 21.0, 27.0, 36.7.)
    pl.token = T <= 4 && k * down_row <= room;
    pl.whole = T * up_row <= room;
    // tokens per item: the MMA's columns, or what fits shared memory, a power of two
    auto cols = [&](int most, bool staged, long long row) {
        int n = most;
        while (n > 1 && staged && (n < T ? n : T) * row > room) n /= 2;
        return n;
    };
    const int up = cols(np == 3 ? 2 : 8, !pl.whole, up_row), down = cols(np == 3 ? 2 : 4, !pl.token, down_row);
    auto log2 = [](int n) { return n == 8 ? 3 : n == 4 ? 2 : n == 2 ? 1 : 0; };
    pl.up_log2 = log2(up);
    pl.down_log2 = log2(down);
    pl.up_cols = up < T ? up : T;
    pl.down_cols = down < T ? down : T;
    const long long up_item = pl.up_cols * up_row, down_item = pl.token ? k * down_row : pl.down_cols * down_row;
    if (room < 0 || (!pl.whole && up_item > room) || down_item > room) return pl;
    auto most = [&](long long item) { return (int)(room / item < kMoeItems ? room / item : kMoeItems); };
    pl.up_items = pl.whole ? kMoeItems : most(up_item);
    pl.down_items = most(down_item);
    long long act = pl.whole ? T * up_row : pl.up_items * up_item;
    if (act < pl.down_items * down_item) act = pl.down_items * down_item;
    if ((long long)S * c.up.RB * sms > UINT32_MAX || (long long)S * c.down.RB * sms > UINT32_MAX) return pl;
    if ((long long)S * c.up.RB * (c.up.KS > c.down.KS ? c.up.KS : c.down.KS) > INT32_MAX || (long long)S * c.down.RB * c.down.KS > INT32_MAX) return pl;
    pl.off_zero = (int)act;
    pl.off_part = pl.off_zero + 16;
    pl.off_ring = pl.off_part + kMoePart;
    pl.off_route = pl.off_ring + ring;
    pl.smem = (size_t)pl.off_route + route;
    pl.blocks = sms;
    auto r256 = [](size_t v) { return (v + 255) / 256 * 256; };
    pl.ws_logits = 256;
    pl.ws_h = pl.ws_logits + r256((size_t)T * ((E + 3) / 4 * 4) * 4);
    pl.ws_part = pl.ws_h + r256((size_t)S * c.down.K * 4);
    pl.workspace = pl.ws_part + (pl.token ? 0 : (size_t)S * c.down.N * 4);
    pl.ok = true;
    return pl;
}

cudaError_t launch_moe_layer(const MoePlan& pl, const MoeCall& c, void* ws, unsigned* err, int stall, int smem_max, cudaStream_t s) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    unsigned* counters = reinterpret_cast<unsigned*>(b);
    float* logits = reinterpret_cast<float*>(b + pl.ws_logits);
    const int E = c.up.E, ldl = (E + 3) / 4 * 4;
    cudaError_t e = launch_pdl_2d(moe_router_kernel, (unsigned)E, (unsigned)((c.T + kRouterTokens - 1) / kRouterTokens), 256, 0, s, c.x, c.xt, c.ldx, c.T, c.up.K, c.router, c.rt, logits, ldl, counters);
    if (e != cudaSuccess) return e;
    MoeParams p;
    p.route = RouteParams();
    p.route.c = c.route;
    p.route.c.logits = logits;
    p.route.c.xt = X_F32;
    p.route.c.ldl = ldl;
    p.route.c.T = c.T;
    p.route.c.E = E;
    p.epl16 = E > 128;
    route_lanes(p.route, p.epl16 ? 16 : 4);
    p.up = c.up;
    p.down = c.down;
    p.x = c.x;
    p.ldx = c.ldx;
    p.xt = c.xt;
    p.h = b + pl.ws_h;
    p.part = reinterpret_cast<float*>(b + pl.ws_part);
    p.y = c.y;
    p.counters = counters;
    p.err = err;
    p.up_log2 = pl.up_log2;
    p.down_log2 = pl.down_log2;
    p.up_cols = pl.up_cols;
    p.down_cols = pl.down_cols;
    p.whole = pl.whole;
    p.up_items = pl.up_items;
    p.down_items = pl.down_items;
    p.off_zero = pl.off_zero;
    p.off_part = pl.off_part;
    p.off_ring = pl.off_ring;
    p.off_route = pl.off_route;
    p.stall = stall;
    return c.xt == X_F16 ? launch_moe_layer_f16(pl, p, smem_max, s) : c.xt == X_BF16 ? launch_moe_layer_bf16(pl, p, smem_max, s) : launch_moe_layer_f32(pl, p, smem_max, s);
}

}  // namespace qmm

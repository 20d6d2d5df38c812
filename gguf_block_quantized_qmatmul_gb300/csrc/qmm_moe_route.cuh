// qmm_moe_route.cuh -- one token's routing, by one warp: qmm_moe_route.cu
// states the mathematics.
#pragma once

#include "qmm_q4g_internal.h"

namespace qmm {

struct RouteParams {
    RouteCall c;
    int tile;              // tokens per tile (a block of the first launch)
    int blocks;            // tiles
    uint8_t* counts;       // [tiles][stride]: slots of each tile by expert (more than one tile)
    int stride;            // bytes from a tile's counts to the next: E rounded up to 16
    int per;               // tiles per block of the second launch
    int vec, vec_bias;     // logits, bias: a lane's experts may be read as vectors
    int group_lanes_log2;  // a group is 2^this lanes' experts; -1: it is not
    unsigned group_magic;  // 2^22 / (experts per group), rounded up: e / group size for e < 512
};

// order-preserving integer key of a float; -0 counts as +0, NaN ranks below -inf; 0 is "none"
__device__ __forceinline__ uint32_t pick_key(float f) {
    if (f != f) return 1u;
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// EPL consecutive values of 4-byte words or fewer, as raw words; vec: they may be read 16 (8, 4) bytes at a time
template <int WORDS>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t w[WORDS]) {
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    } else if constexpr (WORDS == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *p;
    }
}

// One token: EPL consecutive experts per lane.  sk: the warp's row of picks in
// shared memory (groups that are not whole powers of two of lanes).  Lane j <
// top_k returns choice j.
template <int EPL>
__device__ __forceinline__ int route_token(const RouteParams& p, long long tok, uint32_t* sk, int lane) {
    const RouteCall& c = p.c;
    float score[EPL];
    uint32_t key[EPL];
    const long long base = tok * c.ldl;
    const int e0 = lane * EPL;
    float m = -INFINITY;
    // the type is told apart outside of the loads, so that they are in flight together
    if (p.vec) {  // E is a multiple of EPL: a lane has all of its experts or none
        if (c.xt == X_F32) {
            uint32_t w[EPL];
            if (e0 < c.E) load_words<EPL>(reinterpret_cast<const uint32_t*>(static_cast<const float*>(c.logits) + base + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) score[i] = e0 < c.E ? __uint_as_float(w[i]) : -INFINITY;
        } else if constexpr (EPL >= 2) {
            uint32_t w[EPL / 2];
            if (e0 < c.E) load_words<EPL / 2>(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(c.logits) + base + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t h = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
                score[i] = e0 >= c.E ? -INFINITY : c.xt == X_F16 ? h2f(h) : __uint_as_float(h << 16);
            }
        }
    } else if (c.xt == X_F32) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) score[i] = e0 + i < c.E ? static_cast<const float*>(c.logits)[base + e0 + i] : -INFINITY;
    } else {
        uint16_t raw[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) raw[i] = e0 + i < c.E ? static_cast<const uint16_t*>(c.logits)[base + e0 + i] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            score[i] = e0 + i >= c.E ? -INFINITY : c.xt == X_F16 ? h2f(raw[i]) : __uint_as_float((uint32_t)raw[i] << 16);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (score[i] != score[i]) score[i] = -INFINITY;  // a NaN logit is a masked one
        m = fmaxf(m, score[i]);
    }
    if (!c.sigmoid) {
        float total = 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float l = score[i];
            // a row whose mask leaves nothing has no scores; l = m also covers +inf
            const float s = m == -INFINITY ? 0.0f : l == m ? 1.0f : expf(l - m);
            if (!c.bias) key[i] = pick_key(l);
            score[i] = e0 + i < c.E ? s : 0.0f;
            total += score[i];
        }
        if (c.bias || !c.renorm) {
#pragma unroll
            for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            const float d = total > 0.0f ? total : 1.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) score[i] = score[i] / d;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            score[i] = 1.0f / (1.0f + expf(-score[i]));
            if (!c.bias) key[i] = pick_key(score[i]);
        }
    }
    if (c.bias) {
        float b[EPL];
        if (p.vec_bias && e0 < c.E) {
            uint32_t w[EPL];
            load_words<EPL>(reinterpret_cast<const uint32_t*>(c.bias + e0), w);
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = e0 + i < c.E ? c.bias[e0 + i] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = pick_key(score[i] + b[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i >= c.E) key[i] = 0u;
    if (c.groups > 1) {
        uint32_t b1 = 0u, b2 = 0u;  // the two largest picks of this lane's group, in the group's first lane
        int log_lanes;              // lanes per group, a power of two
        if (p.group_lanes_log2 >= 0) {  // a group is whole lanes
            log_lanes = p.group_lanes_log2;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b2 = max(b2, min(b1, key[i]));
                b1 = max(b1, key[i]);
            }
        } else {  // through shared memory: lane r of a group takes its picks r, r + lanes, ...
            const int gs = c.E / c.groups;
            log_lanes = 5;
            while ((c.groups << log_lanes) > 32) --log_lanes;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < c.E) sk[e0 + i] = key[i];
            __syncwarp();
            const int q = lane >> log_lanes;
            if (q < c.groups)
                for (int r = lane & ((1 << log_lanes) - 1); r < gs; r += 1 << log_lanes) {
                    const uint32_t k = sk[q * gs + r];
                    b2 = max(b2, min(b1, k));
                    b1 = max(b1, k);
                }
        }
        for (int o = (1 << log_lanes) >> 1; o; o >>= 1) {
            const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
            b2 = max(max(b2, o2), min(b1, o1));
            b1 = max(b1, o1);
        }
        uint32_t gk = b1;
        if (c.top2 && b2 != 0u) {
            const uint32_t u1 = b1 & 0x80000000u ? b1 & 0x7fffffffu : ~b1, u2 = b2 & 0x80000000u ? b2 & 0x7fffffffu : ~b2;
            gk = pick_key(__uint_as_float(u1) + __uint_as_float(u2));
        }
        if ((lane >> log_lanes) >= c.groups || (lane & ((1 << log_lanes) - 1)) != 0) gk = 0u;
        uint32_t kept = 0u;  // bit per group
        for (int s = 0; s < c.top_groups; ++s) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, gk);
            const int l0 = __ffs(__ballot_sync(0xffffffffu, gk == best)) - 1;
            kept |= 1u << (l0 >> log_lanes);
            if (lane == l0) gk = 0u;
        }
        if (p.group_lanes_log2 >= 0) {
            if (!((kept >> (lane >> log_lanes)) & 1u))
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = 0u;
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (e0 + i < c.E && !((kept >> (((unsigned)(e0 + i) * p.group_magic) >> 22)) & 1u)) key[i] = 0u;
        }
    }
    // the k largest: lane j ends up with choice j (the lowest lane of equals has the lowest expert)
    int my_id = 0;
    float my_score = 0.0f, sum = 0.0f;
    if constexpr (EPL <= 4) {
        // A lane's few experts are put in order first, by pick and then by index; a step is then a reduction, a
        // ballot and a move, some 80 cycles.  (Looking for a lane's largest again after it gave it away: 380 a step.)
        int id[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) id[i] = e0 + i;
#pragma unroll
        for (int n = EPL - 1; n > 0; --n)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool swap = key[i + 1] > key[i];  // equals stay in order
                const uint32_t k0 = key[i];
                const float s0 = score[i];
                const int i0 = id[i];
                key[i] = swap ? key[i + 1] : k0;
                key[i + 1] = swap ? k0 : key[i + 1];
                score[i] = swap ? score[i + 1] : s0;
                score[i + 1] = swap ? s0 : score[i + 1];
                id[i] = swap ? id[i + 1] : i0;
                id[i + 1] = swap ? i0 : id[i + 1];
            }
        for (int j = 0; j < c.top_k; ++j) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
            const int l0 = __ffs(__ballot_sync(0xffffffffu, key[0] == best)) - 1;
            const int got = __shfl_sync(0xffffffffu, id[0], l0);
            const float s = __shfl_sync(0xffffffffu, score[0], l0);
            const bool mine = lane == l0;
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) {
                key[i] = mine ? key[i + 1] : key[i];
                score[i] = mine ? score[i + 1] : score[i];
                id[i] = mine ? id[i + 1] : id[i];
            }
            key[EPL - 1] = mine ? 0u : key[EPL - 1];
            sum += s;
            my_id = lane == j ? got : my_id;
            my_score = lane == j ? s : my_score;
        }
    } else {
        // a lane looks for its own largest again only after it gave it away
        uint32_t b = 0u;
        int bi = 0;
        float bs = 0.0f;
        auto local = [&]() {
            b = 0u;
            bi = 0;
            bs = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const bool more = key[i] > b;
                b = more ? key[i] : b;
                bi = more ? i : bi;
                bs = more ? score[i] : bs;
            }
        };
        local();
        for (int j = 0; j < c.top_k; ++j) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, b);
            const int l0 = __ffs(__ballot_sync(0xffffffffu, b == best)) - 1;
            const int id = __shfl_sync(0xffffffffu, e0 + bi, l0);
            const float s = __shfl_sync(0xffffffffu, bs, l0);
            if (lane == l0) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = i == bi ? 0u : key[i];
                local();
            }
            sum += s;
            if (lane == j) {
                my_id = id;
                my_score = s;
            }
        }
    }
    if (lane < c.top_k) {
        const float v = c.renorm ? (sum > 0.0f ? my_score / sum : 0.0f) : my_score;
        c.ids[tok * c.top_k + lane] = my_id;
        c.weights[tok * c.top_k + lane] = c.scale == 1.0f ? v : v * c.scale;
    }
    return my_id;
}

// What follows from the sizes and alignments of a call (not: tile, blocks, counts, stride, per).
inline void route_lanes(RouteParams& p, int epl) {  // epl: experts per lane
    const RouteCall& c = p.c;
    const int gs = c.E / c.groups;
    p.group_magic = ((1u << 22) + gs - 1) / gs;
    const int bytes = epl * x_size(c.xt), chunk = bytes < 16 ? bytes : 16;
    p.vec = bytes >= 4 && c.E % epl == 0 && (c.ldl * x_size(c.xt)) % chunk == 0 && (reinterpret_cast<uintptr_t>(c.logits) & (chunk - 1)) == 0;
    p.vec_bias = c.bias && c.E % epl == 0 && (reinterpret_cast<uintptr_t>(c.bias) & ((epl < 4 ? epl * 4 : 16) - 1)) == 0;
    p.group_lanes_log2 = -1;
    if (gs % epl == 0 && ((gs / epl) & (gs / epl - 1)) == 0)
        for (p.group_lanes_log2 = 0; (epl << p.group_lanes_log2) < gs;) ++p.group_lanes_log2;
}

}  // namespace qmm

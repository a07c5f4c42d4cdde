// The dropout mask of include/drop.h on the device: Philox4x32-10 (Salmon et
// al. 2011) of a group's counter, 16 bits for each of the group's 8 elements.
//
// A call is 20 widening 32 x 32 products (quarter rate) and 40 xors and adds,
// about 400 cycles of a wavefront for 64 x 8 elements: 3.1e12 elements/s over
// the chip, above what HBM feeds a kernel that reads and writes 4 bytes an
// element (1.2e12 at 5 TB/s), so the mask costs no time of its own beside it.
// 16 bits an element instead of 32 halves the calls; p is then held to 2^-17.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/drop.h"

namespace drop {

// The spec as a kernel takes it: the threshold and scale are the host's, the
// key and offset come from device memory where rng is set.
struct Mask {
    uint64_t seed, offset;
    const drop_rng *rng;
    uint32_t thr;    // kept iff bits >= thr, in [0, 65536]
    float scale;
};

inline Mask mask_of(const drop_spec &s)
{
    Mask m;
    m.seed = s.seed;
    m.offset = s.offset;
    m.rng = s.rng;
    m.thr = (uint32_t)rintf(s.p * 65536.0f);
    m.scale = m.thr >= 65536u ? 0.0f : (float)(65536.0 / (double)(65536u - m.thr));
    return m;
}

// 0, or the DROP_E* of a bad spec (NULL included).
inline int check_spec(const drop_spec *s)
{
    if (!s)
        return DROP_ENULL;
    if (!(s->p >= 0.0f && s->p <= 1.0f) || s->reserved != 0)
        return DROP_EARG;
    if ((uintptr_t)s->rng % 16 != 0)
        return DROP_EALIGN;
    return DROP_OK;
}

struct Key {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ Key key_of(const Mask &m)
{
    uint64_t seed = m.seed, offset = m.offset;
    if (m.rng) {
        seed = m.rng->seed;
        offset = m.rng->offset;
    }
    return Key{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// The group's 128 bits.
__device__ __forceinline__ uint4 bits_of(const Key &key, uint64_t group)
{
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = key.o0, c3 = key.o1;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Element e (0 .. 7) of a group's bits.
__device__ __forceinline__ bool kept(const uint4 &w, int e, uint32_t thr)
{
    const uint32_t x = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
    return ((e & 1) ? x >> 16 : x & 0xFFFFu) >= thr;
}

__device__ __forceinline__ float dropped(float v, const uint4 &w, int e, uint32_t thr, float scale)
{
    return kept(w, e, thr) ? v * scale : 0.0f;
}

}  // namespace drop

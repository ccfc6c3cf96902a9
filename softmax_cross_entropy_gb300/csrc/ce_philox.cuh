// Counter-based random words for dropout: Philox 4x32 with 10 rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", SC 2011). Element i of a tensor takes lane i mod 4 of the block whose
// 128-bit counter is (i div 4) + offset * 2^64 under the 64-bit key `seed`,
// so a word depends on nothing but (seed, offset, i): the backward forms it
// again and no mask is stored.
#pragma once

#include <cstdint>

namespace gbce {

// Which elements dropout keeps, and what it multiplies them by. `state`, two
// int64 on the device, replaces seed and is added to offset when not null
// (a captured graph draws new words by updating it).
struct DropSpec {
    uint64_t seed, offset;
    const int64_t* state;  // {seed, offset} or nullptr
    uint32_t threshold;    // kept when the word is at least floor(p 2^32)
    int mode;              // kDropNone (p = 0), kDropSome, kDropAll (p = 1)
    float scale;           // 1 / (1 - p)
};
enum : int { kDropNone = 0, kDropSome = 1, kDropAll = 2 };

struct PhiloxKey {
    uint32_t k0, k1;  // the seed
    uint32_t o0, o1;  // the offset
};

__device__ __forceinline__ PhiloxKey philox_key(const DropSpec& d) {
    uint64_t seed = d.seed, offset = d.offset;
    if (d.state) {
        seed = static_cast<uint64_t>(d.state[0]);
        offset += static_cast<uint64_t>(d.state[1]);
    }
    return PhiloxKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32),
                     static_cast<uint32_t>(offset), static_cast<uint32_t>(offset >> 32)};
}

// The four words of block `group`.
__device__ __forceinline__ uint4 philox4x32(const PhiloxKey& key, uint64_t group) {
    uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32);
    uint32_t c2 = key.o0, c3 = key.o1;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Dropout of the 4 elements of block `group`: v scaled where kept, else
// exactly 0, whatever v holds (a select: an infinity or NaN that is dropped
// leaves nothing).
__device__ __forceinline__ void drop4(const DropSpec& d, const PhiloxKey& key, uint64_t group,
                                      float* v) {
    const uint4 w = philox4x32(key, group);
    v[0] = w.x >= d.threshold ? v[0] * d.scale : 0.f;
    v[1] = w.y >= d.threshold ? v[1] * d.scale : 0.f;
    v[2] = w.z >= d.threshold ? v[2] * d.scale : 0.f;
    v[3] = w.w >= d.threshold ? v[3] * d.scale : 0.f;
}

}  // namespace gbce

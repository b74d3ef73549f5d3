// Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", SC 2011), and the elements that a dropout keeps by it.
#pragma once

#include <cstdint>

#include "block_internal.h"
#include "model_device.cuh"

namespace fa {

// The four words of one block: ten rounds, each two 32 x 32 bit products whose halves
// change places, on a key that moves by two constants (the rounds' keys are kernel parameters,
// which the exclusive ors take as they are; as sums they were 20 of 82 instructions).
__device__ __forceinline__ uint4 philox(uint64_t lo, uint64_t hi, const uint32_t (*key)[2]) {
    uint32_t c0 = static_cast<uint32_t>(lo), c1 = static_cast<uint32_t>(lo >> 32);
    uint32_t c2 = static_cast<uint32_t>(hi), c3 = static_cast<uint32_t>(hi >> 32);
#pragma unroll
    for (int r = 0; r < kPhiloxRounds; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ key[r][0];
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ key[r][1];
        c1 = static_cast<uint32_t>(b);
        c3 = static_cast<uint32_t>(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint64_t drop_call(const DropArgs &d) {
    return d.offset + (d.counter ? __ldg(reinterpret_cast<const unsigned long long *>(d.counter)) : 0);
}

// Which of a run of eight columns are kept: 16 bits an element, so that one block serves a
// run (32 bits an element would double the ten rounds, which then take as long as the
// memory of 16-bit types).
struct Kept {
    uint32_t w[4];

    __device__ __forceinline__ void draw(const DropArgs &d, uint64_t block, uint64_t call) {
        const uint4 r = philox(block, call, d.key);
        w[0] = r.x;
        w[1] = r.y;
        w[2] = r.z;
        w[3] = r.w;
    }
    // Those of a run that begins ``shift`` columns (1 to 7) before the block's, whose own are here.
    __device__ __forceinline__ void begin_before(const DropArgs &d, uint64_t block, uint64_t call,
                                                 int shift) {
        const uint4 r = philox(block - 1, call, d.key);
        const uint32_t cat[8] = {r.x, r.y, r.z, r.w, w[0], w[1], w[2], w[3]};
        move_down<4>(cat, 16 - 2 * shift, w);
    }
    __device__ __forceinline__ void all() { w[0] = w[1] = w[2] = w[3] = 0xffffffffu; }
    // Zeros in place of the dropped ones of four pairs.
    __device__ __forceinline__ void mask(uint64_t *p, uint32_t threshold) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpair(p[j], lo, hi);
            p[j] = pair((*this)(2 * j, threshold) ? lo : 0.f, (*this)(2 * j + 1, threshold) ? hi : 0.f);
        }
    }
    __device__ __forceinline__ bool operator()(int j, uint32_t threshold) const {
        const uint32_t v = j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16;
        return v >= threshold;
    }
};

}  // namespace fa

// msr_lookback.hpp -- what a tile of a chain does with the words of the tiles
// before it: arithmetic without device builtins or headers (a kernel includes
// it after hip_runtime.h), so that a host program can run it over words of its
// own.
#pragma once

#include <cmath>
#include <cstdint>

namespace msr {

// ---- factors ----------------------------------------------------------------
// A factor f in [0, 1] is held as 1 - f where f >= 1/2 and as -f below (the
// sign bit tells them apart), so that neither a state that hardly decays nor
// one that is nearly gone loses accuracy.  -0 is f = 0.
__device__ __forceinline__ bool far(float z) { return __builtin_bit_cast(int32_t, z) < 0; }
__device__ __forceinline__ float apply(float z, float p) {
    if (!far(z) && __builtin_isinf(p)) return p;  // not p - z p
    return fmaf(-z, p, far(z) ? 0.f : p);
}

// ---- words between tiles ------------------------------------------------------
// Every tile has a word: its pair (f, h), which maps the state p before the tile to f p + h; then (kState) the state after
// it.  A pair whose f is 0 is no state yet: 0 p is NaN where p is not finite.

// factor bits, of NaNs that no factor has, of a word that is not published yet and of one that holds a state
constexpr uint32_t kUnset = 0xffffffffu, kState = 0xfffffffeu;

__device__ __forceinline__ uint64_t pack(uint32_t u, float h) { return (uint64_t)u << 32 | __builtin_bit_cast(uint32_t, h); }
__device__ __forceinline__ uint64_t pair_word(float z, float h) {
    return pack(z != z ? 0x7fc00000u : __builtin_bit_cast(uint32_t, z), h);  // one NaN for all
}
__device__ __forceinline__ uint32_t kind(uint64_t v) { return (uint32_t)(v >> 32); }
__device__ __forceinline__ float value(uint64_t v) { return __builtin_bit_cast(float, (uint32_t)v); }
__device__ __forceinline__ float after(uint64_t v, float p) {  // the state after its stretch
    return kind(v) == kState ? value(v) : apply(__builtin_bit_cast(float, kind(v)), p) + value(v);
}

// The state that a tile starts from: that of the latest of the LOOK tiles before it whose state is known, and the pairs
// since.  word(i) is the word of the tile i + 1 before it (of the chain's first where there is none), pause() is called
// between polls.  Which state that is depends on how far the other workgroups are; the result does not, since every tile's
// end state is formed from its start state by the same pair.  NaN after `spins` polls without one, so that it shows in all
// that follows.
template <int LOOK, typename Word, typename Pause>
__device__ __forceinline__ float look_back(int spins, const Word &word, const Pause &pause) {
    uint64_t v[LOOK];
    int from = -1;  // the latest state with no word missing after it
    for (int spin = 0; spin < spins; ++spin) {
#pragma unroll
        for (int i = 0; i < LOOK; ++i) v[i] = word(i);
        bool open = false;
#pragma unroll
        for (int i = 0; i < LOOK; ++i) {
            if (from < 0 && !open && kind(v[i]) == kState) from = i;
            open = open || kind(v[i]) == kUnset;
        }
        if (from >= 0) break;
        pause();
    }
    float p = __builtin_nanf("");
#pragma unroll
    for (int i = LOOK - 1; i >= 0; --i)
        if (i <= from) p = after(v[i], p);
    return p;
}

}  // namespace msr

// rope.cuh -- device helpers shared by the kernels that turn feature pairs by their
// position (rope.cu, norm_rope.cu): a feature in fp32, and sine and cosine of an angle
// that is held as a fraction of a turn.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace spa {

__device__ __forceinline__ float up(float x) { return x; }
__device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }

// Sine and cosine of the angle pos * advance, in units of 2^-64 turns, modulo one turn.
__device__ __forceinline__ void sincos_of(unsigned long long advance, int pos, float& s, float& c) {
  const unsigned long long turn =
      static_cast<unsigned long long>(static_cast<long long>(pos)) * advance;
  // signed fraction of a turn in [-1/2, 1/2): angle / pi = 2 * fraction.  Its first 24
  // bits as a float, without rounding; the next 24 turn the result by the angle that is
  // left, below pi 2^-23, whose square is nothing here.
  const float half_turns = static_cast<float>(static_cast<int>(turn >> 32) & ~0xff) * 0x1p-31f;
  const float rest = static_cast<float>(static_cast<uint32_t>(turn >> 16) & 0xffffffu) * (3.14159265f * 0x1p-47f);
  float s0, c0;
  sincospif(half_turns, &s0, &c0);
  s = fmaf(rest, c0, s0);
  c = fmaf(-rest, s0, c0);
}

}  // namespace spa

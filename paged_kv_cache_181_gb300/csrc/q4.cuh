// The 4-bit pool record: one (block, head) of 16 tokens x D channels in 10 * D bytes.
//   codes  [16 tokens][D/2 bytes]   channel c in byte c/2, even channels in the low nibble
//   pairs  [16 tokens][D/32 groups] (fp16 step, fp16 low); a code n stands for fp16(step * n + low)
// One record is contiguous, so a block of one head is one 1280-byte (D = 128) piece of memory for the kernels
// that read it, and a token's codes are one 64-byte piece for the kernel that writes them.  Groups of 32
// channels: 5 bits a value; one pair for a whole 128-channel row would be 4.25, but a single large channel
// then widens the steps of all of them.
#pragma once

#include "common.cuh"

template <int D>
struct Q4 {
  static constexpr int kRowBytes = D / 2;            // codes of one token
  static constexpr int kGroups = D / 32;             // pairs of one token
  static constexpr int kPairs = 16 * kRowBytes;      // offset of the pairs in a record
  static constexpr int kRecord = kPairs + 16 * kGroups * 4;
};

// Eight codes of one word (channel i at bits 4i) as fp16 pairs: h[i] = (n_i, n_{i+4}), exact.
// 0x6400 is 1024 in fp16, whose last bit is worth 1: or-ing a nibble into the low bits gives 1024 + n, and one
// four bits higher 1024 + 16 n.
PKV_DEVINLINE __half2 q4_pick(uint32_t w, uint32_t mask) {
  // (w & mask) | 0x64006400 in one instruction: with both constants as immediates it would be two.
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x64006400u));
  return *reinterpret_cast<__half2*>(&d);
}
PKV_DEVINLINE void q4_unpack(uint32_t w, __half2 (&h)[4]) {
  const __half2 k1024 = __half2half2(__ushort_as_half(0x6400));
  const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00)), k64 = __half2half2(__ushort_as_half(0xd400));  // 1/16, -64
  h[0] = __hsub2(q4_pick(w, 0x000f000fu), k1024);
  h[1] = __hfma2(q4_pick(w, 0x00f000f0u), sixteenth, k64);
  w >>= 8;
  h[2] = __hsub2(q4_pick(w, 0x000f000fu), k1024);
  h[3] = __hfma2(q4_pick(w, 0x00f000f0u), sixteenth, k64);
}

// The eight fp16 values of a word under one pair, as h[i] = (value_i, value_{i+4}).
PKV_DEVINLINE void q4_values(uint32_t w, __half2 pair, __half2 (&h)[4]) {
  q4_unpack(w, h);
  const __half2 step = __low2half2(pair), low = __high2half2(pair);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __hfma2(h[i], step, low);
}

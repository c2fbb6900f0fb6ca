// Loads from memory straight into LDS, and the barriers around them.
#pragma once

#include "device.h"

namespace moe {

// A buffer offset past every resource: the load reads zeros and makes no
// memory request. Resources are kept shorter than this.
constexpr uint32_t kPastEnd = 0xFFFFFFF0u;
constexpr size_t kMostBytes = 0xFFFFF000u;

// A buffer resource over `bytes` bytes from `base`; offsets at or past the end
// read zeros.
__device__ __forceinline__ u32x4 buffer_over(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// The same in every lane, for the compiler too.
__device__ __forceinline__ u32x4 uniform(const u32x4& v) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)v[i]);
  return r;
}

// One load of 64 x 16 bytes by the whole wave: lane i's 16 bytes at offset
// voff + soff of the resource go to LDS byte lds + 16 i. As asm, so that the
// compiler does not track the LDS writes (it would wait for every load in
// flight before each LDS read): the kernels wait for their own loads (vmcnt)
// and meet the block before anyone reads what they wrote.
//
// The scalar operands may come from v_readfirstlane, and a load must be five
// wait states behind the vector instruction that wrote a scalar register it
// reads; the compiler does not look into the asm, so the wait stands there
// (s_nop 4 is five states, one of which m0 needs too). m0, where the load takes
// its LDS address from, is an operand: the compiler sets it and knows.
__device__ __forceinline__ void dma16(const u32x4& rs, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile(
      "s_nop 4\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "{m0}"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(voff), "s"(uniform(rs)), "s"(__builtin_amdgcn_readfirstlane((int)soff))
      : "memory");
}

// Two of them behind one wait, the second to the 1 KB that follows. ONCE: for
// data that is read once (it does not displace what the caches hold for others).
template <bool ONCE>
__device__ __forceinline__ void dma16_two(const u32x4& rs, uint32_t lds, uint32_t v0, uint32_t v1,
                                          uint32_t soff) {
  int m = __builtin_amdgcn_readfirstlane((int)lds);
  const u32x4 r = uniform(rs);
  const int s = __builtin_amdgcn_readfirstlane((int)soff);
  if (ONCE)
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %1, %3, %4 offen nt lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen nt lds"
        : "+{m0}"(m)
        : "v"(v0), "v"(v1), "s"(r), "s"(s)
        : "memory", "scc");
  else
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %1, %3, %4 offen lds\n\t"
        "s_add_u32 m0, m0, 0x400\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds"
        : "+{m0}"(m)
        : "v"(v0), "v"(v1), "s"(r), "s"(s)
        : "memory", "scc");
}

// N loads to consecutive KB from `lds` on.
template <bool ONCE, int N>
__device__ __forceinline__ void dma16_run(const u32x4& rs, uint32_t lds, const uint32_t (&voff)[N],
                                          uint32_t soff) {
  static_assert(N % 2 == 0 || !ONCE, "single loads keep what they read");
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) dma16_two<ONCE>(rs, lds + j * 1024u, voff[j], voff[j + 1], soff);
  if (N % 2) dma16(rs, lds + (N - 1) * 1024u, voff[N - 1], soff);
}

// One load with 4 bytes a lane.
__device__ __forceinline__ void dma4(const u32x4& rs, uint32_t lds, uint32_t voff) {
  asm volatile(
      "s_nop 4\n\t"
      "buffer_load_dword %1, %2, 0 offen lds"
      :
      : "{m0}"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(voff), "s"(uniform(rs))
      : "memory");
}

// Until the wave's LDS operations are done. (Not as asm: the compiler would not
// know, and wait once more, in the next stage, before it writes to a register
// that an LDS read of this one returned to.)
__device__ __forceinline__ void wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0) alone
  asm volatile("" ::: "memory");
}

// Until at most n of the wave's vector memory operations are in flight.
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(n) : "memory");
}

// 16 bytes a lane from byte `at` of `base` (resource rs; at = kPastEnd: zeros),
// of any alignment. The load's range check drops the whole dword that the
// array's end cuts: where `edge` says that a lane may reach byte `end`, such
// lanes take their bytes one by one, after every load in flight. Bytes from the
// end on are zeros or what was there.
__device__ __forceinline__ void dma16_bytes(const u32x4& rs, const uint8_t* base, uint32_t end,
                                            uint32_t lds, uint32_t at, int lane, bool edge) {
  if (__builtin_expect(!edge, 1)) {
    dma16(rs, lds, at, 0);
    return;
  }
  const bool cut = at < end && end - at < 16 && ((end - at) & 3) != 0;
  dma16(rs, lds, cut ? kPastEnd : at, 0);
  wait_loads<0>();
  typedef __attribute__((address_space(3))) uint8_t* Lds;
  if (cut)
    for (uint32_t b = 0; at + b < end; ++b) *reinterpret_cast<Lds>(lds + lane * 16 + b) = base[at + b];
  wait_lds();
}

// Whether a lane that reads `bytes` bytes from `first` on, 16 at a time, may
// reach an array's end at a byte that is no whole dword behind its place.
__device__ __forceinline__ bool at_edge(uint32_t first, uint32_t bytes, uint32_t end) {
  return __any(first < end && end - first < bytes + 16 && ((end - first) & 3) != 0);
}

// The block meets; LDS reads and writes stay on their side.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace moe

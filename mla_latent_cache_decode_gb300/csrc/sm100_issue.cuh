// Forms of the tensor-core instructions for the prompt kernels' loops: MMAs by
// the low words of their descriptors, and names for what a load has written.
#pragma once
#include "sm100.cuh"

namespace mla {
namespace sm100 {

// After tmem_wait_ld: 32 (16) registers that a load wrote.  The wait itself names
// no register, so nothing else keeps the compiler from moving what uses them
// ahead of it.  No instruction.
__device__ __forceinline__ void tmem_loaded32(uint32_t *r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_loaded16(uint32_t *r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]));
}

// Of the 64 bits only the address field, in the low word, changes in an issue
// loop.  The MMAs below take low words and one constant high word (a stride of
// 1,024 bytes between groups of eight rows, 128-byte swizzle): half the address
// arithmetic and registers.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
__device__ __forceinline__ uint32_t desc_low(const void *p, uint32_t lbo_bytes) {
  // (in a cluster the address carries the CTA's rank above its 18 bits)
  return (smem_u32(p) >> 4 & 0x3FFFu) | (lbo_bytes >> 4 << 16);
}
// D (+)= A B, A and B in shared memory; A in tensor memory.
__device__ __forceinline__ void mma_ss_low(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t more) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(more), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts_low(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t more) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(more), "n"(kDescHigh)
      : "memory");
}

}  // namespace sm100
}  // namespace mla

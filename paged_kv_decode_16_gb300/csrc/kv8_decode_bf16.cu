// kv8_decode_bf16.cu -- bf16 instantiations of the 8-bit cache's decode kernel.
#include "kv8_decode.cuh"

namespace pkv {

Kv8DecodeInfo kv8_decode_info_bf16(int head_dim, int rows) {
    return pick_kv8_decode_info<__nv_bfloat16>(head_dim, rows);
}

}  // namespace pkv

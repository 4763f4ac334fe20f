// kv8_decode_f16.cu -- f16 instantiations of the 8-bit cache's decode kernel.
#include "kv8_decode.cuh"

namespace pkv {

Kv8DecodeInfo kv8_decode_info_f16(int head_dim, int rows) {
    return pick_kv8_decode_info<__half>(head_dim, rows);
}

}  // namespace pkv

// library.cu -- the library's one translation unit: the BitLinear entry points
// and those of the key/value cache share the device status word, the wait limit
// and the host helpers.
#include "bitnet.cu"

#include "kv.cuh"

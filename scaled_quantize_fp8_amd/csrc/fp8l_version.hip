// Identity of the library: the ABI version and the hash of the sources it was
// built from, in a translation unit of its own so that only this one depends
// on every source.
#include "../../include/fp8linear.h"

#ifndef FP8L_SOURCE_HASH
#define FP8L_SOURCE_HASH "unknown"
#endif

extern "C" {
int fp8_abi_version(void) { return FP8_ABI_VERSION; }
const char* fp8_source_hash(void) { return FP8L_SOURCE_HASH; }
}

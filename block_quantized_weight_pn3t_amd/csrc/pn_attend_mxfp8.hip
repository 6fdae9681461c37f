// pn_attend_mxfp8.hip -- the attention kernels over MXFP8 caches.
#include "pn_attend.h"

namespace pn {
PN_ATTEND_FORMAT(PN_CACHE_MXFP8)
}  // namespace pn
